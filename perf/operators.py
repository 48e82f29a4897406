"""Cases of the dense feed-forward operators: the gated block of the dense layers, its backward
pass, and the projection shared by many requests with a low-rank adapter of each beside it.

    gated_ffn            h = act(x Wg^T) * (x Wu^T)
    gated_ffn_backward   dx, dWg, dWu from x, Wg, Wu and dh (g and u computed again)
    adapter_proj         y = x W^T + s_a (x A_a^T) B_a^T + residual, a = the token's adapter or none

``run`` computes each in its plain form (32 bits, one rounding of each output) or, with ``own``,
through the package's calls. Activations and weights are BF16, row-major; a linear weight is
[out, in]. Adapters: A [n, rank, in], B [n, out, rank], one FP32 scale each; ids int32 per token,
-1 for a token without one.
"""
import math

import torch

own = False

ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
BF16 = torch.bfloat16
_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # a toy layer's decode of four tokens: launch latency only
        {"name": "gated tiny T4", "op": "gated_ffn", "T": 4, "H": 512, "I": 384, "act": "silu"},
        # batch-1 decode through a dense layer of the 24B stack's width: the weights' bytes
        {"name": "gated decode T1", "op": "gated_ffn", "T": 1, "H": 2048, "I": 7168, "act": "silu"},
        # decode of 96 requests at once: still the weights' bytes, on the tensor cores
        {"name": "gated batch T96", "op": "gated_ffn", "T": 96, "H": 2048, "I": 7168, "act": "silu"},
        # a ragged prefill chunk at sizes that fill no tile
        {"name": "gated ragged T777", "op": "gated_ffn", "T": 777, "H": 1000, "I": 2840, "act": "gelu_tanh"},
        # a long prefill chunk: the matrix products
        {"name": "gated prefill T8192", "op": "gated_ffn", "T": 8192, "H": 2048, "I": 7168, "act": "silu"},
        # fine-tuning a short odd batch with the exact GELU: small products, weight gradients' bytes
        {"name": "backward ragged T205", "op": "gated_ffn_backward", "T": 205, "H": 1416, "I": 2008, "act": "gelu"},
        # the gradient of a block of an expert's size over a common batch
        {"name": "backward T2048", "op": "gated_ffn_backward", "T": 2048, "H": 2048, "I": 1536, "act": "silu"},
        # a training micro-batch of the dense layer: the largest work
        {"name": "backward T8192", "op": "gated_ffn_backward", "T": 8192, "H": 2048, "I": 7168, "act": "silu"},
        # batch-1 decode of the down projection with one adapter of a pool
        {"name": "adapters decode T1", "op": "adapter_proj", "T": 1, "K": 7168, "N": 2048, "rank": 16,
         "adapters": 8, "runs": False},
        # 64 requests decoding, nearly each with an adapter of its own
        {"name": "adapters batch T64", "op": "adapter_proj", "T": 64, "K": 7168, "N": 2048, "rank": 16,
         "adapters": 48, "runs": False},
        # ragged prefill of a few requests at sizes that fill no tile, an odd rank
        {"name": "adapters ragged T531", "op": "adapter_proj", "T": 531, "K": 1352, "N": 1048, "rank": 24,
         "adapters": 5, "runs": True},
        # a long prefill chunk of many requests one after another
        {"name": "adapters prefill T8192", "op": "adapter_proj", "T": 8192, "K": 7168, "N": 2048, "rank": 32,
         "adapters": 24, "runs": True},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["gated_ffn", "gated_ffn_backward", "adapter_proj"])
    most = max(work(c)["flops"] for c in listed())
    while True:
        T, a, b = _log(rng, 1, 8192), _log(rng, 256, 4096, 8), _log(rng, 256, 8192, 8)
        if op == "adapter_proj":
            c = {"op": op, "T": T, "K": b, "N": a, "rank": rng.choice([8, 16, 16, 24, 32, 40, 64, 128]),
                 "adapters": _log(rng, 1, 64), "runs": rng.random() < 0.5}
            plain = 2.0 * T * c["adapters"] * c["rank"] * (a + b)  # the plain form's adapter products
        else:
            c = {"op": op, "T": T, "H": a, "I": b, "act": rng.choice(sorted(ACTS))}
            plain = 0.0
        if work(c)["flops"] + plain <= most:
            return c


def _normal(gen, shape, std):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(BF16)


def _ids(case, gen):
    """One adapter id per token: each token its own request, or runs of tokens of one request."""
    T, n = case["T"], case["adapters"]
    if case["runs"]:
        # request boundaries at random places, about one request per adapter
        cuts = torch.rand(T, generator=gen, device="cuda") < n / T
        request = torch.cumsum(cuts.to(torch.int64), 0)
        of_request = torch.randint(-1, n, (T + 1,), generator=gen, device="cuda")
        return of_request[request].to(torch.int32)
    return torch.randint(-1, n, (T,), generator=gen, device="cuda").to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "adapter_proj":
        T, K, N, r, n = (case[k] for k in ("T", "K", "N", "rank", "adapters"))
        s["x"] = _normal(gen, (T, K), 0.5)
        s["w"] = _normal(gen, (N, K), 0.02)
        s["residual"] = _normal(gen, (T, N), 1.0)
        s["lora_a"] = _normal(gen, (n, r, K), K ** -0.5)
        s["lora_b"] = _normal(gen, (n, N, r), 0.3 * r ** -0.5)
        s["scale"] = torch.rand(n, generator=gen, device="cuda") * 1.5 + 0.5
        s["ids"] = _ids(case, gen)
        return s
    T, H, I = case["T"], case["H"], case["I"]
    s["x"] = _normal(gen, (T, H), 1.0)  # a normalised layer input
    s["w_gate"] = _normal(gen, (I, H), H ** -0.5)
    s["w_up"] = _normal(gen, (I, H), H ** -0.5)
    if case["op"] == "gated_ffn_backward":
        s["dh"] = _normal(gen, (T, I), 0.01)
    return s


# ---------------------------------------------------------------- plain form

def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(_C0 * (g + _C1 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(_C0 * (g + _C1 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * g * g)


def _plain(s):
    x = s["x"].float()
    if s["op"] == "adapter_proj":
        n, r, K = s["lora_a"].shape
        N = s["w"].shape[0]
        ids = s["ids"].long()
        # every adapter's inner product, of which a token keeps its own
        v = (x @ s["lora_a"].float().view(n * r, K).t()).view(-1, n, r) * s["scale"].view(1, n, 1)
        mine = ids.view(-1, 1) == torch.arange(n, device=ids.device)
        v = torch.where(mine.unsqueeze(2), v, torch.zeros_like(v)).view(-1, n * r)
        b = s["lora_b"].float().permute(0, 2, 1).reshape(n * r, N)
        return {"y": (x @ s["w"].float().t() + v @ b + s["residual"].float()).to(BF16)}
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg.t(), x @ wu.t()
    if s["op"] == "gated_ffn":
        return {"h": (_act(g, s["act"]) * u).to(BF16)}
    dh = s["dh"].float()
    dg, du = dh * u * _act_grad(g, s["act"]), dh * _act(g, s["act"])
    return {"dx": (dg @ wg + du @ wu).to(BF16), "dw_gate": (dg.t() @ x).to(BF16), "dw_up": (du.t() @ x).to(BF16)}


def run(state):
    s = state
    if not own:
        return _plain(s)
    import packed_mxfp4_w4a16_b200 as moe
    if s["op"] == "gated_ffn":
        return {"h": moe.moe_gated_ffn(s["x"], s["w_gate"], s["w_up"], ACTS[s["act"]])}
    if s["op"] == "gated_ffn_backward":
        dx, dwg, dwu = moe.moe_gated_ffn_backward(s["x"], s["w_gate"], s["w_up"], s["dh"], ACTS[s["act"]])
        return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
    return {"y": moe.moe_adapter_proj(s["x"], s["w"], s["lora_a"], s["lora_b"], s["scale"], s["ids"],
                                      residual=s["residual"])}


def work(case):
    if case["op"] == "adapter_proj":
        T, K, N, r, n = (case[k] for k in ("T", "K", "N", "rank", "adapters"))
        # about T n / (n + 1) tokens have an adapter; as many adapters as those can name
        draws = min(T, n + 1) if case["runs"] else T
        used = n * (1.0 - (1.0 - 1.0 / (n + 1)) ** draws)
        withone = T * n / (n + 1.0)
        return {"bytes": 2.0 * (T * K + N * K + 2 * T * N) + 4.0 * T + used * (2.0 * r * (K + N) + 4.0),
                "flops": 2.0 * T * K * N + 2.0 * withone * r * (K + N)}
    T, H, I = case["T"], case["H"], case["I"]
    if case["op"] == "gated_ffn":
        return {"bytes": 2.0 * (T * H + 2 * I * H + T * I), "flops": 4.0 * T * H * I}
    return {"bytes": 2.0 * (2 * T * H + 4 * I * H + T * I), "flops": 12.0 * T * H * I}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in FP64: gradients by differentiating the block, adapters one at a time."""
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "adapter_proj":
        y = s["residual"].double() + x @ s["w"].double().t()
        for a in sorted(set(s["ids"].tolist()) - {-1}):
            rows = torch.nonzero(s["ids"] == a).flatten()
            inner = x[rows] @ s["lora_a"][a].double().t()
            y[rows] += float(s["scale"][a]) * (inner @ s["lora_b"][a].double().t())
        return {"y": y}
    leaves = [x, s["w_gate"].double(), s["w_up"].double()]
    grads = case["op"] == "gated_ffn_backward"
    for t in leaves:
        t.requires_grad_(grads)
    f = torch.nn.functional
    gate, up = f.linear(leaves[0], leaves[1]), f.linear(leaves[0], leaves[2])
    if case["act"] == "silu":
        h = f.silu(gate) * up
    else:
        h = f.gelu(gate, approximate="tanh" if case["act"] == "gelu_tanh" else "none") * up
    if not grads:
        return {"h": h}
    dx, dwg, dwu = torch.autograd.grad(h, leaves, s["dh"].double())
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
