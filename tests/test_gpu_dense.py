"""The dense feed-forward operators on the GPU against FP64, element by
element, at the sizes and inputs where they can go wrong."""
import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from dense_util import (ACTS, adapter64, assert_within, gated64, gated_backward64, normal)

pytestmark = pytest.mark.gpu

# tokens: single ones, either side of the small-batch limit and of a tile, odd ones
TOKENS = [1, 2, 7, 8, 9, 16, 33, 127, 128, 129, 257, 600]
# (H, I): the smallest, not multiples of a tile or of 64, the 24B layer's
SHAPES = [(8, 8), (72, 40), (200, 136), (512, 384), (1000, 520), (2048, 1536)]


def gated_inputs(T, H, I, seed=0):
    return (normal((T, H), 1.0, seed), normal((I, H), H ** -0.5, seed + 1),
            normal((I, H), H ** -0.5, seed + 2))


@pytest.fixture(autouse=True)
def no_status():
    yield
    assert moe.moe_dense_status() == 0


@pytest.mark.parametrize("H,I", SHAPES)
@pytest.mark.parametrize("T", TOKENS)
def test_gated_forward(T, H, I):
    x, wg, wu = gated_inputs(T, H, I, seed=T)
    act = sorted(ACTS)[T % 3]
    h = moe.moe_gated_ffn(x, wg, wu, ACTS[act])
    assert_within(h, *gated64(x, wg, wu, act), f"h {T}x{H}x{I} {act}")


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("T", [3, 200])
def test_gated_forward_large_gates(act, T):
    """Gates far into both tails of the activation."""
    x, wg, wu = gated_inputs(T, 256, 264, seed=5)
    h = moe.moe_gated_ffn(x, wg * 30, wu, ACTS[act])
    assert_within(h, *gated64(x, wg * 30, wu, act), f"h {act}")


@pytest.mark.parametrize("H,I", SHAPES)
@pytest.mark.parametrize("T", [1, 7, 8, 9, 64, 65, 130, 300])
def test_gated_backward(T, H, I):
    x, wg, wu = gated_inputs(T, H, I, seed=T + 100)
    dh = normal((T, I), 0.1, T + 50)
    act = sorted(ACTS)[(T + I // 8) % 3]
    got = moe.moe_gated_ffn_backward(x, wg, wu, dh, ACTS[act])
    want, bound = gated_backward64(x, wg, wu, dh, act)
    for g, w, b, what in zip(got, want, bound, ("dx", "dw_gate", "dw_up")):
        assert_within(g, w, b, f"{what} {T}x{H}x{I} {act}")


@pytest.mark.parametrize("act", sorted(ACTS))
def test_gated_backward_against_differences(act):
    """The FP64 gradient formulas against central differences of the FP64
    forward (the kernels are held to the formulas by the test above)."""
    x, wg, wu = (t.double() for t in gated_inputs(3, 16, 24, seed=9))
    dh = normal((3, 24), 1.0, 3).double()
    (dx, dwg, dwu), _ = gated_backward64(x, wg, wu, dh, act)
    eps = 1e-5

    def loss(a, b, c):
        return float((gated64(a, b, c, act)[0] * dh).sum())

    for which, grad in ((0, dx), (1, dwg), (2, dwu)):
        args = [x, wg, wu]
        for flat in range(0, grad.numel(), 7):
            d = torch.zeros_like(args[which]).view(-1)
            d[flat] = eps
            d = d.view_as(args[which])
            up = loss(*[a + d if i == which else a for i, a in enumerate(args)])
            dn = loss(*[a - d if i == which else a for i, a in enumerate(args)])
            assert abs((up - dn) / (2 * eps) - float(grad.view(-1)[flat])) < 1e-6


@pytest.mark.parametrize("T,H,I,act", [(2600, 1800, 1304, "silu"), (2561, 2048, 1536, "gelu_tanh"),
                                       (4000, 1288, 72, "gelu")])
def test_gated_many_tokens(T, H, I, act):
    """Enough 256-row tiles for the CTA pairs, ragged and full, several per pair."""
    x, wg, wu = gated_inputs(T, H, I, seed=T)
    h = moe.moe_gated_ffn(x, wg, wu, ACTS[act])
    assert_within(h, *gated64(x, wg, wu, act), f"h {T}x{H}x{I} {act}")
    dh = normal((T, I), 0.1, T + 50)
    got = moe.moe_gated_ffn_backward(x, wg, wu, dh, ACTS[act])
    want, bound = gated_backward64(x, wg, wu, dh, act)
    for g, w, b, what in zip(got, want, bound, ("dx", "dw_gate", "dw_up")):
        assert_within(g, w, b, f"{what} {T}x{H}x{I} {act}")


def test_gated_backward_parts_alone():
    x, wg, wu = gated_inputs(70, 136, 200, seed=1)
    dh = normal((70, 200), 0.1, 2)
    dx, dwg, dwu = moe.moe_gated_ffn_backward(x, wg, wu, dh)
    only = moe.moe_gated_ffn_backward(x, wg, wu, dh, need_dw=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = moe.moe_gated_ffn_backward(x, wg, wu, dh, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dwg) and torch.equal(only[2], dwu)


def test_no_tokens():
    wg = normal((40, 24), 1.0, 0)
    x = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    assert moe.moe_gated_ffn(x, wg, wg).shape == (0, 40)
    dwg, dwu = torch.ones_like(wg), torch.ones_like(wg)
    dx, dwg, dwu = moe.moe_gated_ffn_backward(x, wg, wg, x.new_empty(0, 40), dw_gate=dwg, dw_up=dwu)
    assert dx.shape == (0, 24) and not dwg.any() and not dwu.any()
    assert moe.moe_adapter_proj(x, wg).shape == (0, 40)


def test_rms_norm_flag():
    for T, H in ((1, 64), (5, 2048), (200, 1000)):
        r, wg, wu = gated_inputs(T, H, 136, seed=T)
        r = r * 3
        xn = torch.empty_like(r)
        h = moe.moe_gated_ffn(r, wg, wu, flags=moe.FFN_RMSNORM, x_norm=xn)
        r64 = r.double()
        want = r64 / torch.sqrt((r64 * r64).mean(1, keepdim=True) + 1e-6)
        # FP32 sum of squares, square root, division, product: H + 8 roundings
        bound = (2.0 ** -8 + (H + 8) * 2.0 ** -24) * want.abs() * 1.01 + 2.0 ** -133
        assert_within(xn, want, bound, "x_norm")
        assert torch.equal(h, moe.moe_gated_ffn(xn, wg, wu))


# ------------------------------------------------------------- adapters

def adapter_inputs(T, K, N, rank, n, runs, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ids = torch.randint(-1, n, (T,), generator=gen, device="cuda", dtype=torch.int32)
    if runs:
        ids = ids.sort().values[torch.arange(T, device="cuda") // 1]
        ids = ids.roll(T // 3).contiguous()
    return dict(x=normal((T, K), 0.5, seed + 1), w=normal((N, K), 0.02, seed + 2),
                lora_a=normal((n, rank, K), K ** -0.5, seed + 3),
                lora_b=normal((n, N, rank), 0.3 * rank ** -0.5, seed + 4),
                lora_scale=torch.rand(n, generator=gen, device="cuda") * 1.5 + 0.5,
                adapter_ids=ids, residual=normal((T, N), 1.0, seed + 5))


def check_adapter(d, what, **kw):
    y = moe.moe_adapter_proj(**d, **kw)
    want, bound = adapter64(d["x"], d["w"], d.get("lora_a"), d.get("lora_b"), d.get("lora_scale"),
                            d.get("adapter_ids"), d.get("residual"))
    assert_within(y, want, bound, what)
    return y


@pytest.mark.parametrize("T,H,I", [(2600, 1032, 2568), (5000, 1032, 520), (2561, 520, 1032)])
def test_gated_last_wave_of_half_tiles(T, H, I):
    """Few tiles over a whole number of waves, and columns that end inside a half tile."""
    x, wg, wu = gated_inputs(T, H, I, seed=T)
    assert_within(moe.moe_gated_ffn(x, wg, wu), *gated64(x, wg, wu, "silu"), "h")
    dh = normal((T, I), 0.1, T + 5)
    want, bound = gated_backward64(x, wg, wu, dh, "silu")
    for got, w, b, name in zip(moe.moe_gated_ffn_backward(x, wg, wu, dh), want, bound, ("dx", "dwg", "dwu")):
        assert_within(got, w, b, name)


PROJ = [(8, 8, 8, 1), (136, 72, 24, 3), (384, 512, 16, 20), (1000, 520, 64, 7), (1536, 2048, 16, 40),
        (2048, 264, 40, 5), (264, 392, 136, 4), (512, 256, 256, 3)]


@pytest.mark.parametrize("K,N,rank,n", PROJ)
@pytest.mark.parametrize("T", TOKENS)
def test_adapter_proj(T, K, N, rank, n):
    check_adapter(adapter_inputs(T, K, N, rank, n, runs=T % 2 == 1, seed=T), f"y {T} {K} {N} {rank} {n}")


@pytest.mark.parametrize("T,K,N,rank,n,runs", [(2600, 520, 1800, 16, 9, True), (2561, 264, 2048, 40, 30, False),
                                               (5000, 136, 1032, 128, 3, True)])
def test_adapter_proj_many_tokens(T, K, N, rank, n, runs):
    d = adapter_inputs(T, K, N, rank, n, runs, seed=T)
    check_adapter(d, f"y {T} {K} {N} {rank} {n}")
    check_adapter({"x": d["x"], "w": d["w"], "residual": d["residual"]}, "plain")


@pytest.mark.parametrize("T,K,N,rank,n,runs", [(1285, 344, 2056, 8, 1, True), (1300, 136, 2048, 40, 64, False),
                                               (1290, 72, 2048, 16, 1024, False), (1290, 72, 2048, 8, 1032, False),
                                               (2049, 200, 1800, 24, 100, True), (2600, 72, 5368, 24, 5, False),
                                               (2600, 72, 5160, 136, 3, True), (200, 72, 64, 8, 1024, False),
                                               (200, 72, 64, 8, 1025, False)])
def test_adapter_proj_large_pools(T, K, N, rank, n, runs):
    """Long batches whose tiles name many adapters, and pools on both sides of
    the size up to which a tile lists them from a bitmap."""
    check_adapter(adapter_inputs(T, K, N, rank, n, runs, seed=T), f"y {T} {K} {N} {rank} {n}")


@pytest.mark.parametrize("rank", [24, 136])
def test_bad_adapter_in_a_long_batch(rank):
    T, N = 1300, 2056
    d = adapter_inputs(T, 136, N, rank, 5, False, seed=rank)
    whole = {k: v.clone() for k, v in d.items()}
    clean = moe.moe_adapter_proj(**d)
    mine = d["adapter_ids"] == 1
    touched = torch.zeros(N, dtype=torch.bool, device="cuda")
    touched[[0, 300, N - 1]] = True
    d["lora_b"][1, touched, rank - 1] = float("inf")
    y = moe.moe_adapter_proj(**d)
    assert torch.equal(y[~mine], clean[~mine]) and torch.equal(y[mine][:, ~touched], clean[mine][:, ~touched])
    assert not torch.isfinite(y[mine][:, touched]).any()
    d["lora_a"][1, 2, 9] = float("nan")
    y = moe.moe_adapter_proj(**d)
    assert torch.equal(y[~mine], clean[~mine]) and not torch.isfinite(y[mine]).any()
    d["adapter_ids"][mine] = 5
    y = moe.moe_adapter_proj(**d)
    assert moe.moe_dense_status() == moe.DEVICE_BAD_ADAPTER_ID
    # (not the bits of `clean`: without adapter 1 the others' ranks share their
    # steps of 16 products with other zeros, which is another order of one FP32 sum)
    want, bound = adapter64(whole["x"], whole["w"], whole["lora_a"], whole["lora_b"], whole["lora_scale"],
                            whole["adapter_ids"], whole["residual"])
    assert_within(y[~mine], want[~mine], bound[~mine], "others")
    assert torch.equal(y[mine], moe.moe_adapter_proj(d["x"], d["w"], residual=d["residual"])[mine])


@pytest.mark.parametrize("T", [1, 5, 8, 40, 200])
def test_plain_projection(T):
    d = adapter_inputs(T, 520, 264, 8, 1, False, seed=T)
    check_adapter({"x": d["x"], "w": d["w"], "residual": d["residual"]}, "with residual")
    check_adapter({"x": d["x"], "w": d["w"]}, "without")


@pytest.mark.parametrize("T", [1, 6, 24, 150])
def test_adapter_none_and_residual_in_place(T):
    d = adapter_inputs(T, 328, 200, 16, 4, False, seed=T)
    d["adapter_ids"].fill_(-1)
    plain = moe.moe_adapter_proj(d["x"], d["w"], residual=d["residual"])
    assert torch.equal(moe.moe_adapter_proj(**d), plain)
    r = d.pop("residual").clone()
    assert torch.equal(moe.moe_adapter_proj(**d, residual=r, y=r), plain)


@pytest.mark.parametrize("T", [1, 7, 20, 129, 300])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_bad_adapter_reaches_its_own_tokens_only(T, value):
    """Tokens of other adapters, and those without one, keep their bits; in
    the tokens of the bad one, exactly the touched outputs are not finite."""
    d = adapter_inputs(T, 264, 136, 16, 3, False, seed=T)
    d["adapter_ids"][T // 2] = 1
    clean = moe.moe_adapter_proj(**d)
    mine = d["adapter_ids"] == 1
    d["lora_b"][1, 5, 3] = value
    d["lora_b"][1, 77, 0] = value
    y = moe.moe_adapter_proj(**d)
    assert torch.equal(y[~mine], clean[~mine])
    finite = torch.isfinite(y[mine])
    keep = torch.ones(136, dtype=torch.bool, device="cuda")
    keep[5] = keep[77] = False
    assert finite[:, keep].all() and not finite[:, ~keep].any()
    assert torch.equal(y[mine][:, keep], clean[mine][:, keep])
    d["lora_a"][1, 2, 9] = value
    y = moe.moe_adapter_proj(**d)
    assert torch.equal(y[~mine], clean[~mine])
    assert not torch.isfinite(y[mine]).any()


@pytest.mark.parametrize("T", [3, 20, 150])
def test_bad_token_reaches_its_own_row_only(T):
    d = adapter_inputs(T, 264, 136, 16, 3, False, seed=T + 1)
    clean = moe.moe_adapter_proj(**d)
    d["x"][T // 2, 7] = float("nan")
    y = moe.moe_adapter_proj(**d)
    rows = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[T // 2]).all()
    x, wg, wu = gated_inputs(T, 264, 136, seed=3)
    clean = moe.moe_gated_ffn(x, wg, wu)
    x[T // 2, 7] = float("inf")
    h = moe.moe_gated_ffn(x, wg, wu)
    assert torch.equal(h[rows], clean[rows])


@pytest.mark.parametrize("T", [4, 60])
def test_adapter_ids_out_of_range(T):
    d = adapter_inputs(T, 136, 72, 8, 3, False, seed=T)
    none = dict(d, adapter_ids=torch.full_like(d["adapter_ids"], -1))
    want = moe.moe_adapter_proj(**none)
    assert moe.moe_dense_status() == 0
    for bad in (3, -2, 2 ** 31 - 1, -2 ** 31):
        d["adapter_ids"].fill_(bad)
        assert torch.equal(moe.moe_adapter_proj(**d), want)
        assert moe.moe_dense_status() == moe.DEVICE_BAD_ADAPTER_ID
