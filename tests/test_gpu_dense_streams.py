"""Dense calls on a stream that is not the current one: what they allocate."""
import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from dense_util import adapter64, assert_within, gated64, gated_backward64, normal

pytestmark = pytest.mark.gpu

MARK = 7.0


class PendingWork:
    """Blocks of given sizes (in BF16 elements) that the current stream has freed
    on the host while its work on them is still to come: each is copied, and then
    overwritten, behind a wait of some ten milliseconds.  A call on another stream
    that is handed such a block destroys the copy, or has its own data destroyed."""

    def __init__(self, sizes):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        blocks = [torch.full((n,), MARK, dtype=torch.bfloat16, device="cuda") for n in sizes]
        self.copies = [torch.empty_like(b) for b in blocks]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        for b, c in zip(blocks, self.copies):
            c.copy_(b)
            b.zero_()

    def check(self):
        torch.cuda.synchronize()
        for c in self.copies:
            assert (c == MARK).all(), "a call on another stream wrote into memory of pending work"


@pytest.mark.parametrize("T", [4, 600])
def test_new_outputs_wait_for_no_work_of_the_current_stream(T):
    H, I, rank = 1024, 1536, 16
    x, wg, wu = normal((T, H), 1, 1), normal((I, H), 0.03, 2), normal((I, H), 0.03, 3)
    dh, wd = normal((T, I), 0.1, 4), normal((H, I), 0.03, 5)
    a, b, sc = normal((3, rank, I), 0.03, 6), normal((3, H, rank), 0.1, 7), torch.ones(3, device="cuda")
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 3
    # load the kernels: a first launch may wait for the device
    h0 = moe.moe_gated_ffn(x, wg, wu)
    moe.moe_gated_ffn_backward(x, wg, wu, dh)
    moe.moe_adapter_proj(h0, wd, a, b, sc, ids)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    pending = PendingWork([T * I])
    h = moe.moe_gated_ffn(x, wg, wu, stream=side)
    pending.check()
    assert_within(h, *gated64(x, wg, wu, "silu"), "h")

    pending = PendingWork([T * H, I * H, I * H, 2 * T * I])
    got = moe.moe_gated_ffn_backward(x, wg, wu, dh, stream=side)
    pending.check()
    want, bound = gated_backward64(x, wg, wu, dh, "silu")
    for g, w, e, what in zip(got, want, bound, ("dx", "dw_gate", "dw_up")):
        assert_within(g, w, e, what)

    words = moe.moe_adapter_proj_workspace_bytes(T, I, H, 3, rank) // 2
    pending = PendingWork([T * H, words])
    y = moe.moe_adapter_proj(h0, wd, a, b, sc, ids, stream=side)
    pending.check()
    want, bound = adapter64(h0, wd, a, b, sc, ids, None)
    assert_within(y, want, bound, "y")


def test_outputs_outlive_their_readers_on_the_current_stream():
    """An output of a call on another stream, read by the current one and let go:
    the next call's output may not take its place before the reader is done."""
    x, wg, wu = normal((512, 1024), 1, 1), normal((1536, 1024), 0.03, 2), normal((1536, 1024), 0.03, 3)
    side = torch.cuda.Stream()
    want = moe.moe_gated_ffn(x, wg, wu)
    other = moe.moe_gated_ffn(-x, wg, wu)
    nx = -x
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        h = moe.moe_gated_ffn(x, wg, wu, stream=side)
        copy = torch.empty_like(h)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(50_000_000)
        copy.copy_(h)
        del h
        again = moe.moe_gated_ffn(nx, wg, wu, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(copy, want) and torch.equal(again, other)


@pytest.mark.parametrize("T", [3, 300])
def test_a_captured_branch_on_another_stream(T):
    """Calls on a second stream that takes part in a capture: a graph of two
    branches whose outputs and workspaces come from the graph's memory."""
    x, wg, wu = normal((T, 264), 1, 1), normal((328, 264), 0.06, 2), normal((328, 264), 0.06, 3)
    dh, wd = normal((T, 328), 0.1, 4), normal((264, 328), 0.05, 5)
    a, b, sc = normal((5, 24, 328), 0.05, 6), normal((5, 264, 24), 0.05, 7), torch.ones(5, device="cuda")
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 6 - 1

    def branch(stream):
        h = moe.moe_gated_ffn(x, wg, wu, stream=stream)
        return [h, moe.moe_adapter_proj(h, wd, a, b, sc, ids, stream=stream),
                *moe.moe_gated_ffn_backward(x, wg, wu, dh, stream=stream)]

    want = branch(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        first = branch(side)
        second = branch(None)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in first + second:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for out in (first, second):
            assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert moe.moe_dense_status() == 0


@pytest.mark.parametrize("T", [4, 600])
def test_buffers_of_a_layer_wait_for_no_work_of_the_current_stream(T):
    """The buffers that a layer allocates when it is made, used on another stream."""
    H, I, rank = 1024, 1536, 16
    x, wg, wu, wd = normal((T, H), 1, 1), normal((I, H), 0.03, 2), normal((I, H), 0.03, 3), normal((H, I), 0.03, 5)
    lora = (normal((3, rank, I), 0.03, 6), normal((3, H, rank), 0.1, 7), torch.ones(3, device="cuda"))
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 3
    want = moe.DenseFFN(wg, wu, wd, lora=lora, max_tokens=T).forward(x, ids, rmsnorm=True)
    side = torch.cuda.Stream()
    words = moe.moe_adapter_proj_workspace_bytes(T, I, H, 3, rank) // 2
    pending = PendingWork([T * I, T * H, words])
    layer = moe.DenseFFN(wg, wu, wd, lora=lora, max_tokens=T)
    y = layer.forward(x, ids, rmsnorm=True, stream=side)
    pending.check()
    assert torch.equal(y, want)
