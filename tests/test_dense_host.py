"""Host-side checks of the dense feed-forward calls: they refuse bad
arguments before anything touches a GPU."""
import ctypes as C

import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe

ARG, OK = -1, 0


@pytest.fixture(scope="module")
def lib():
    return moe.load()


# addresses that are never read: every call below is refused (or does nothing)
X, WG, WU, H_, XN, DH, DX, DG, DU, WS = (C.c_void_p(0x10000000 * (i + 1)) for i in range(10))


def test_gated_ffn_refusals(lib):
    def call(x=X, T=4, H=64, I=32, wg=WG, wu=WU, act=0, flags=0, xn=None, h=H_):
        return lib.moe_gated_ffn(x, T, H, I, wg, wu, act, flags, xn, h, None)
    for bad in (dict(T=-1), dict(T=2 ** 30 + 1), dict(H=0), dict(H=12), dict(H=65544), dict(I=4), dict(I=-8), dict(act=3),
                dict(act=-1), dict(flags=2), dict(flags=1), dict(xn=XN), dict(h=X), dict(h=WG), dict(h=WU),
                dict(flags=1, xn=H_), dict(flags=1, xn=X), dict(h=C.c_void_p(X.value + 16))):
        assert call(**bad) == ARG, bad
    assert call(T=0) == OK
    assert call(T=0, x=None, h=None) == OK


def test_backward_refusals(lib):
    def call(x=X, T=4, H=64, I=32, wg=WG, wu=WU, act=0, dh=DH, dx=DX, dg=DG, du=DU, ws=WS, n=1 << 20):
        return lib.moe_gated_ffn_backward(x, T, H, I, wg, wu, act, dh, dx, dg, du, ws, n, None)
    for bad in (dict(T=-1), dict(T=2 ** 31 - 1), dict(H=4), dict(I=20), dict(act=7), dict(dg=None), dict(du=None),
                dict(dx=None, dg=None, du=None), dict(dx=X), dict(dg=DU), dict(du=WU), dict(dx=DH),
                dict(ws=X), dict(ws=DX), dict(T=0, dg=DG, du=DG)):
        assert call(**bad) == ARG, bad
    assert call(T=0, dg=None, du=None) == OK
    n = C.c_size_t()
    assert lib.moe_gated_ffn_backward_workspace_bytes(3, 64, 40, C.byref(n)) == OK and n.value == 512
    assert lib.moe_gated_ffn_backward_workspace_bytes(0, 64, 40, C.byref(n)) == OK and n.value == 256
    assert lib.moe_gated_ffn_backward_workspace_bytes(3, 63, 40, C.byref(n)) == ARG
    assert lib.moe_gated_ffn_backward_workspace_bytes(3, 64, 40, None) == ARG
    # past 32 bits
    assert lib.moe_gated_ffn_backward_workspace_bytes(1 << 20, 64, 65536, C.byref(n)) == OK
    assert n.value == 4 * (1 << 20) * 65536


def test_adapter_refusals(lib):
    a, b, s, ids, y, r = (C.c_void_p(0x200000000 + 0x10000000 * i) for i in range(6))

    def call(x=X, T=4, K=64, N=32, w=WG, res=None, n=2, rank=8, a=a, b=b, s=s, ids=ids, y=y, ws=WS,
             size=1 << 20):
        return lib.moe_adapter_proj(x, T, K, N, w, res, n, rank, a, b, s, ids, y, ws, size, None)
    for bad in (dict(T=-1), dict(T=2 ** 30 + 1), dict(K=60), dict(N=4), dict(n=-1), dict(rank=0), dict(rank=12),
                dict(rank=264), dict(n=0), dict(y=X), dict(y=WG), dict(y=a), dict(y=b), dict(y=WS),
                dict(res=C.c_void_p(y.value + 16)), dict(res=WS), dict(ws=X), dict(ws=ids)):
        assert call(**bad) == ARG, bad
    assert call(T=0) == OK
    n = C.c_size_t()
    assert lib.moe_adapter_proj_workspace_bytes(9, 64, 32, 0, 0, C.byref(n)) == OK and n.value == 0
    assert lib.moe_adapter_proj_workspace_bytes(9, 64, 32, 2, 8, C.byref(n)) == OK and n.value > 0
    assert lib.moe_adapter_proj_workspace_bytes(9, 64, 32, 2, 9, C.byref(n)) == ARG
    assert lib.moe_dense_status(None, None) == ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the refusal of a host without a GPU")
def test_no_device(lib):
    v = C.c_uint()
    assert lib.moe_dense_status(None, C.byref(v)) != OK
    assert lib.moe_gated_ffn(X, 4, 64, 32, WG, WU, 0, 0, None, H_, None) != OK


def test_binding_refuses_host_tensors_shapes_and_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_gated_ffn(x, w, w), lambda: moe.moe_gated_ffn(x, None, w),
                 lambda: moe.moe_gated_ffn(None, w, w),
                 lambda: moe.moe_gated_ffn_backward(x, w, w, x), lambda: moe.moe_adapter_proj(x, w),
                 lambda: moe.moe_adapter_proj(x, w, lora_a=x)):
        with pytest.raises(moe.MoEError):
            call()
