"""Dense layers as they are used: DenseFFN, stacks of dense and MoE layers, CUDA
graphs, streams, calls that share or must not share buffers."""
import os
import subprocess
import sys

import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from dense_util import adapter64, assert_within, gated64, gated_backward64, normal
from gpu_util import dev_layer
from workloads import synth

pytestmark = pytest.mark.gpu


def make_dense(H, I, T, lora=None, seed=0, act=0):
    wg, wu = normal((I, H), H ** -0.5, seed), normal((I, H), H ** -0.5, seed + 1)
    wd = normal((H, I), I ** -0.5, seed + 2)
    if lora is not None:
        n, rank = lora
        lora = (normal((n, rank, I), I ** -0.5, seed + 3), normal((n, H, rank), 0.3 * rank ** -0.5, seed + 4),
                torch.linspace(0.5, 2, n, device="cuda"))
    return moe.DenseFFN(wg, wu, wd, act, lora, max_tokens=T)


def make_stack(dense, n_moe, T, persistent=None, seed=3):
    shape = synth.TINY
    weights = [dev_layer(synth.make_layer(shape, seed=seed, layer=l)) for l in range(n_moe)]
    return moe.MoEStack(dense + weights, shape.E, shape.H, shape.I, shape.top_k, T=T, persistent=persistent)


@pytest.mark.parametrize("T", [1, 8, 9, 40, 300])
def test_dense_layer_stage_by_stage(T):
    L = make_dense(512, 392, T, lora=(3, 16), seed=T)
    x, r = normal((T, 512), 1, 50), normal((T, 512), 1, 51)
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 4 - 1
    y = L.forward(x, ids, residual=r)
    assert_within(L.h[:T], *gated64(x, L.w_gate, L.w_up, "silu"), "h")
    want, bound = adapter64(L.h[:T], L.w_down, *L.lora, ids, r)
    assert_within(y, want, bound, "y")
    assert torch.equal(L(x), moe.moe_adapter_proj(L.h[:T], L.w_down))
    dh = normal((T, 392), 0.1, 5)
    got = L.gated_backward(x, dh)
    want, bound = gated_backward64(x, L.w_gate, L.w_up, dh, "silu")
    for g, w, b in zip(got, want, bound):
        assert_within(g, w, b, "gradient")
    with pytest.raises(moe.MoEError):
        L.forward(torch.cat([x, x]))
    assert L.status() == 0


@pytest.mark.parametrize("T", [1, 5, 12])
def test_stack_of_dense_and_moe_layers(T):
    """The stack's step is the dense layers' calls and then moe_layer_ex, bit
    for bit, eager and replayed, with adapters named before each replay."""
    H = synth.TINY.H
    dense = [make_dense(H, 264, T, lora=(4, 8), seed=10), make_dense(H, 512, T, seed=20)]
    st = make_stack(dense, 2, T)
    assert (st.stack is not None) == (T == 1)
    r0 = normal((T, H), 1, 77)
    outs = {}
    for ids in (-1, 2):
        want = r0.clone()
        st.adapter_ids.fill_(ids)
        for L in dense:
            want = L.forward(want, st.adapter_ids, residual=want, rmsnorm=True)
        xn = torch.empty_like(want)
        for L in st.moe_layers:
            kid = torch.empty(T, 4, dtype=torch.int32, device="cuda")
            kw = torch.empty(T, 4, dtype=torch.float32, device="cuda")
            moe.moe_layer_ex(L.handle, want, L.router_w, L.router_b, moe.ROUTE_RMSNORM, xn, None, kid, kw, want,
                             want, 0)
        st.r.copy_(r0)
        st.enqueue()
        assert torch.equal(st.r, want)
        st.r.copy_(r0)
        st.enqueue_layers()
        assert torch.equal(st.r, want)
        for _ in range(2):
            st.r.copy_(r0)
            st.step()
            torch.cuda.synchronize()
            assert torch.equal(st.r, want)
        outs[ids] = want
    assert not torch.equal(outs[-1], outs[2])
    assert st.status() == 0
    st.close()


def test_stack_with_a_dense_layer_between():
    """Dense layers elsewhere than ahead: layer by layer, never one launch."""
    H = synth.TINY.H
    weights = [dev_layer(synth.make_layer(synth.TINY, seed=1, layer=l)) for l in range(2)]
    layers = [weights[0], make_dense(H, 128, 1), weights[1]]
    s = synth.TINY
    st = moe.MoEStack(layers, s.E, s.H, s.I, s.top_k)
    assert st.stack is None
    st.r.copy_(normal((1, H), 1, 1))
    st.step()
    torch.cuda.synchronize()
    assert torch.isfinite(st.r).all() and st.status() == 0
    st.close()
    with pytest.raises(moe.MoEError):
        moe.MoEStack(layers, s.E, s.H, s.I, s.top_k, persistent=True)
    with pytest.raises(moe.MoEError):  # another H
        moe.MoEStack([make_dense(H + 8, 128, 1)], s.E, s.H, s.I, s.top_k)
    with pytest.raises(moe.MoEError):  # buffers of fewer tokens
        moe.MoEStack([make_dense(H, 128, 1)], s.E, s.H, s.I, s.top_k, T=2)


def all_calls(T, seed):
    """Inputs and one pass of every operator, with outputs of its own."""
    x, wg, wu = normal((T, 264), 1, seed), normal((328, 264), 0.06, seed + 1), normal((328, 264), 0.06, seed + 2)
    dh, wd = normal((T, 328), 0.1, seed + 3), normal((264, 328), 0.05, seed + 4)
    a, b = normal((5, 24, 328), 0.05, seed + 5), normal((5, 264, 24), 0.05, seed + 6)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) * 7 % 6) - 1
    scale = torch.ones(5, device="cuda")

    def run(stream=None):
        h = moe.moe_gated_ffn(x, wg, wu, 2, stream=stream)
        y = moe.moe_adapter_proj(h, wd, a, b, scale, ids, residual=x, stream=stream)
        return [h, y, *moe.moe_gated_ffn_backward(x, wg, wu, dh, 1, stream=stream)]

    return run


@pytest.mark.parametrize("T", [3, 20, 700])
def test_same_bits_again_on_another_stream_and_in_graphs(T):
    run = all_calls(T, T)
    want = run()
    torch.cuda.synchronize()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(s)  # the stream as an argument, another one current
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs, replayed in turn and again
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for k in (0, 1, 1, 0):
        for t in graphs[k][1]:
            t.zero_()
        graphs[k][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[k][1], want))
    assert moe.moe_dense_status() == 0


@pytest.mark.parametrize("T", [2, 150])
def test_calls_on_two_streams_at_once(T):
    """Calls without shared buffers may overlap."""
    runs = [all_calls(T, 11), all_calls(T, 22)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for k in (0, 1):
            got[k].append(runs[k](streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


@pytest.mark.parametrize("T", [1, 30])
def test_one_workspace_for_calls_in_order(T):
    """Nothing in a workspace outlives a call: other contents, other shapes
    and NaN before it change nothing."""
    a, b, sc = normal((3, 16, 136), 0.1, 1), normal((3, 72, 16), 0.1, 2), torch.ones(3, device="cuda")
    x, w = normal((T, 136), 1, 3), normal((72, 136), 0.1, 4)
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 3
    want = moe.moe_adapter_proj(x, w, a, b, sc, ids)
    ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(moe.moe_adapter_proj(x, w, a, b, sc, ids, workspace=ws), want)
        moe.moe_gated_ffn_backward(x, w, w, normal((T, 72), 1, 5), workspace=ws)


def test_workspace_and_output_refusals():
    x, w = normal((20, 136), 1, 3), normal((72, 136), 0.1, 4)
    dh = normal((20, 72), 1, 5)
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    odd = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")[8:]
    for ws, code in ((small, -5), (odd, -4)):
        with pytest.raises(moe.MoEError) as e:
            moe.moe_gated_ffn_backward(x, w, w, dh, workspace=ws)
        assert e.value.code == code
    with pytest.raises(moe.MoEError):  # not contiguous
        moe.moe_gated_ffn(normal((20, 272), 1, 3)[:, :136], w, w)
    with pytest.raises(moe.MoEError):  # another type
        moe.moe_gated_ffn(x.half(), w, w)
    with pytest.raises(moe.MoEError):  # an output over an input
        moe.moe_gated_ffn(x, w, w, h=x.view(-1)[:20 * 72].view(20, 72))
    big = normal((21, 136), 1, 3)
    with pytest.raises(moe.MoEError) as e:  # rows that start off 16 bytes
        moe.moe_gated_ffn(big.view(-1)[4:4 + 20 * 136].view(20, 136), w, w)
    assert e.value.code == -4
    host = torch.zeros(20, 136, dtype=torch.bfloat16)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_gated_ffn(host, w, w)
    assert e.value.code == -3


def test_outputs_behind_the_last_row_stay():
    """Rows of a larger buffer behind the T of the call are left as they were."""
    for T in (1, 6, 13, 130, 257):
        x, wg, wu = normal((T, 264), 1, T), normal((136, 264), 0.06, 1), normal((136, 264), 0.06, 2)
        h = torch.full((T + 3, 136), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_gated_ffn(x, wg, wu, h=h[:T])
        assert (h[T:] == 7).all() and not (h[:T] == 7).all()
        dx = torch.full((T + 3, 264), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_gated_ffn_backward(x, wg, wu, h[:T].clone(), dx=dx[:T])
        assert (dx[T:] == 7).all()
        y = torch.full((T + 3, 264), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_adapter_proj(h[:T], normal((264, 136), 0.1, 3), y=y[:T])
        assert (y[T:] == 7).all()


def test_more_than_32_bits_of_elements():
    """Offsets past 2^31 elements, in h and in dg | du: the last rows of a long
    batch get the bits of the same rows alone."""
    T, H, I = 70000, 8, 32768
    x = normal((T, H), 1, 0)
    wg, wu = normal((I, H), 0.3, 1), normal((I, H), 0.3, 2)
    h = moe.moe_gated_ffn(x, wg, wu)
    assert torch.equal(h[-300:], moe.moe_gated_ffn(x[-300:].contiguous(), wg, wu))
    dx, _, _ = moe.moe_gated_ffn_backward(x, wg, wu, h, need_dw=False)
    want, bound = gated_backward64(x[-40:], wg, wu, h[-40:], "silu")
    assert_within(dx[-40:], want[0], bound[0], "dx")


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="a second GPU")
def test_memory_of_another_device_is_refused():
    w = normal((72, 136), 0.1, 4)
    with pytest.raises(moe.MoEError):
        moe.moe_gated_ffn(normal((20, 136), 1, 3, device="cuda:1"), w, w)


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
import packed_mxfp4_w4a16_b200 as moe
T = {T}
n = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
x, wg, wu, dh, wd = n(T, 512), n(264, 512), n(264, 512), n(T, 264), n(512, 264)
a, b, sc = n(3, 16, 264), n(3, 512, 16), torch.ones(3, device="cuda")
ids = torch.zeros(T, dtype=torch.int32, device="cuda")

def run():
    h = moe.moe_gated_ffn(x, wg, wu)
    y = moe.moe_adapter_proj(h, wd, a, b, sc, ids, residual=x)
    return [h, y, *moe.moe_gated_ffn_backward(x, wg, wu, dh)]

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(out, run()))
assert moe.moe_dense_status() == 0
"""


@pytest.mark.parametrize("T", [1, 30, 4000])
def test_first_call_of_a_process_may_be_captured(T):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root, T=T)], capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
