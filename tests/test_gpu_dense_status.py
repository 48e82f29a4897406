"""The status word of the dense calls: nothing set is lost."""
import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from dense_util import normal

pytestmark = pytest.mark.gpu


def test_no_status_bit_is_lost_while_the_word_is_read():
    """A bit that another stream sets at any moment of a read is returned by that
    read or by the next one."""
    x, w = normal((4, 136), 1, 1), normal((72, 136), 0.1, 2)
    a, b, sc = normal((3, 8, 136), 0.1, 3), normal((3, 72, 8), 0.1, 4), torch.ones(3, device="cuda")
    ids = torch.full((4,), 3, dtype=torch.int32, device="cuda")
    y = torch.empty(4, 72, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_adapter_proj_workspace_bytes(4, 136, 72, 3, 8), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    moe.moe_dense_status()
    lost = 0
    for i in range(4000):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200 * (i % 400))  # up to 40 us
        moe.moe_adapter_proj(x, w, a, b, sc, ids, y=y, workspace=ws, stream=side)
        seen = moe.moe_dense_status()
        side.synchronize()
        seen |= moe.moe_dense_status()
        lost += seen != moe.DEVICE_BAD_ADAPTER_ID
    assert lost == 0, f"{lost} of 4000 bits lost"


def test_readers_in_several_threads_take_each_bit_once():
    """Threads that read at the same time: a bit goes to exactly one of them."""
    import threading

    x, w = normal((4, 136), 1, 1), normal((72, 136), 0.1, 2)
    a, b, sc = normal((3, 8, 136), 0.1, 3), normal((3, 72, 8), 0.1, 4), torch.ones(3, device="cuda")
    ids = torch.full((4,), 3, dtype=torch.int32, device="cuda")
    moe.moe_adapter_proj(x, w, a, b, sc, ids)
    torch.cuda.synchronize()
    moe.moe_dense_status()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(50):
        moe.moe_adapter_proj(x, w, a, b, sc, ids)
        torch.cuda.synchronize()
        seen = [None] * 4
        start = threading.Barrier(4)

        def read(k):
            start.wait()
            seen[k] = moe.moe_dense_status(streams[k])

        threads = [threading.Thread(target=read, args=(k,)) for k in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(seen) == [0, 0, 0, moe.DEVICE_BAD_ADAPTER_ID]


def test_a_reader_waits_for_its_own_stream_only():
    """While one thread waits for a busy stream, another reads on an idle one."""
    import threading

    moe.moe_dense_status()
    busy, idle = torch.cuda.Stream(), torch.cuda.Stream()
    moe.moe_dense_status(idle)
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(4_000_000_000)  # about two seconds
    entered = threading.Event()

    def read():
        entered.set()
        moe.moe_dense_status(busy)

    t = threading.Thread(target=read)
    t.start()
    entered.wait()
    threading.Event().wait(0.2)  # well into the other's wait
    moe.moe_dense_status(idle)
    assert t.is_alive()
    t.join()
