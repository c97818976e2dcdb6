"""The operators of a feed-forward layer, as cases that can be timed and compared.

Four operators: a linear layer with bias, activation and residual in one kernel, the gated pair of linear layers
(both projections, the activation and the product in one kernel), and the backward pass of each.  With ``own`` false
``run`` computes them with elementary torch operations in FP32, with ``own`` true through ``bf16_gemm_skinny_gb300``.

n tokens, M output features, K input features; W [M, K], x [n, K], everything 16-bit (BF16 or FP16).

linear            z = x W^T + b,  y = act(z) + r;                        y, and z where it is kept for the backward pass
gated             g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) * u;    h, and g and u where they are kept
linear_backward   dz = dy * act'(z);  dx = dz W,  dW = dz^T x,  db = sum over the tokens of dz
gated_backward    dg = dh * u * act'(g),  du = dh * act(g);  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dbg, dbu

The kept z, g and u are inputs of the backward passes as they were rounded.  Gradients have the inputs' type, those of
the weights and biases FP32 where ``grad32`` is set.
"""
import math
import random

import torch

own = False

NAMES = ("op", "type", "act", "n", "M", "K", "bias", "residual", "keep", "grad32", "pad")


def _case(name, *values):
    return dict(zip(NAMES, values), name=name)


def listed():
    return [
        # one user's token through the gate and up projections: the stream of the weights
        _case("gated_decode_one", "gated", "bf16", "silu", 1, 17408, 5120, False, False, False, False, 0),
        # a batch of tokens, one of each request
        _case("gated_decode_batch", "gated", "bf16", "silu", 24, 17408, 5120, False, False, False, False, 0),
        # a short prompt through a small model's layer, odd feature count, trained (g and u are kept)
        _case("gated_chunk_odd", "gated", "f16", "gelu_tanh", 333, 2731, 1024, True, False, True, False, 0),
        # a prompt's chunk through a large model's layer
        _case("gated_prefill", "gated", "bf16", "silu", 4096, 17408, 5120, False, False, False, False, 0),
        # the projection back down of one token, onto the residual stream
        _case("linear_decode_one", "linear", "bf16", "none", 1, 5120, 17408, False, True, False, False, 0),
        # a few drafted tokens through a small layer: pure latency
        _case("linear_small", "linear", "f16", "gelu", 4, 1000, 1024, True, False, False, False, 0),
        # rows of odd length, so that no row but the first starts on a boundary
        _case("linear_ragged", "linear", "bf16", "relu", 777, 1031, 4099, True, False, True, False, 0),
        # the projection back down of a prompt's chunk
        _case("linear_prefill", "linear", "bf16", "none", 4096, 5120, 17408, False, True, False, False, 0),
        # training step of an output projection, gradients of the weights in FP32
        _case("linear_backward_train", "linear_backward", "bf16", "none", 8192, 5120, 4096, True, False, False, True, 0),
        # a small layer with an activation, x a part of wider rows
        _case("linear_backward_small", "linear_backward", "f16", "gelu", 200, 1000, 1024, True, False, False, False, 64),
        # training step of a small model's gated layer, odd sizes
        _case("gated_backward_mid", "gated_backward", "f16", "gelu_tanh", 1500, 2731, 1000, True, False, False, False, 8),
        # training step of a large model's gated layer: the largest
        _case("gated_backward_train", "gated_backward", "bf16", "silu", 4096, 17408, 5120, False, False, False, False, 0),
    ]


def draw(rng: random.Random):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("linear", "gated", "linear_backward", "gated_backward"))
    c = {"op": op, "type": rng.choice(("bf16", "f16")), "act": rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))}
    if op.startswith("gated") and c["act"] == "none":
        c["act"] = "silu"
    step = rng.choice((1, 8, 64))          # sizes of any remainder, of whole vectors, of whole tiles
    while True:
        c["n"] = log(1, 8192) if op in ("linear", "gated") else log(16, 8192)
        c["M"] = max(step, log(64, 17408) // step * step)
        c["K"] = max(step, log(64, 17408) // step * step)
        if c["M"] * c["K"] <= 17408 * 5120 and c["n"] * c["M"] <= 4096 * 17408 and c["n"] * c["M"] * c["K"] <= 4096 * 17408 * 5120:
            break
    c["bias"] = rng.random() < 0.5
    c["residual"] = op == "linear" and rng.random() < 0.5
    c["keep"] = op in ("linear", "gated") and rng.random() < 0.3
    c["grad32"] = op == "linear_backward" and c["act"] == "none"
    c["pad"] = rng.choice((0, 0, 8, 64))
    return {k: c[k] for k in NAMES}


def _type(c):
    return torch.bfloat16 if c["type"] == "bf16" else torch.float16


def prepare(case, seed):
    c, t = case, _type(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, m, k = c["n"], c["M"], c["K"]

    def normal(*shape, size=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=t).mul_(size)

    # normalised activations, each channel with a size of its own; x is the first part of wider rows where pad is set
    rows = normal(n, k + c["pad"]) * torch.exp(0.4 * torch.randn(k + c["pad"], generator=g, device="cuda")).to(t)
    st = {"case": c, "x": rows[:, :k], "x_stride": k + c["pad"], "w": [normal(m, k, size=k ** -0.5) for _ in range(2 if "gated" in c["op"] else 1)]}
    st["b"] = [normal(m, size=0.2) for _ in st["w"]] if c["bias"] else [None] * len(st["w"])

    def empty(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if c["op"] in ("linear", "gated"):
        st["r"] = normal(n, m, size=2.0) if c["residual"] else None
        st["out"] = empty(n, m)
        st["kept"] = [empty(n, m) for _ in st["w"]] if c["keep"] else [None] * len(st["w"])
    else:
        # what the forward pass kept, and the gradient from above
        st["kept"] = [st["x"] @ w.T if b is None else st["x"] @ w.T + b for w, b in zip(st["w"], st["b"])]
        st["dy"] = normal(n, m, size=0.05)
        gt = torch.float32 if c["grad32"] else t
        st["dx"] = empty(n, k)
        st["dw"] = [empty(m, k, dtype=gt) for _ in st["w"]]
        st["db"] = [empty(m, dtype=gt) if c["bias"] else None for _ in st["w"]]
    return st


ROOT_2_OVER_PI = math.sqrt(2 / math.pi)


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(ROOT_2_OVER_PI * (z + 0.044715 * z * z * z)))
    return z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        v = torch.tanh(ROOT_2_OVER_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + v) + 0.5 * z * (1 - v * v) * ROOT_2_OVER_PI * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain(st):
    c, t = st["case"], _type(st["case"])
    x, w = st["x"].float(), [a.float() for a in st["w"]]
    if c["op"] in ("linear", "gated"):
        z = [x @ a.T if b is None else x @ a.T + b.float() for a, b in zip(w, st["b"])]
        y = _act(c["act"], z[0])
        if c["op"] == "gated":
            y = y * z[1]
        elif c["residual"]:
            y = y + st["r"].float()
        return [y.to(t)] + ([a.to(t) for a in z] if c["keep"] else [])
    z, dy = [a.float() for a in st["kept"]], st["dy"].float()
    if c["op"] == "gated_backward":
        dz = [dy * z[1] * _slope(c["act"], z[0]), dy * _act(c["act"], z[0])]
    else:
        dz = [dy * _slope(c["act"], z[0])]
    gt = torch.float32 if c["grad32"] else t
    dx = sum(d @ a for d, a in zip(dz, w))
    return [dx.to(t)] + [(d.T @ x).to(gt) for d in dz] + ([d.sum(0).to(gt) for d in dz] if c["bias"] else [])


def _own(st):
    import bf16_gemm_skinny_gb300 as bsk

    c = st["case"]
    kind = bsk.TYPE_BF16 if c["type"] == "bf16" else bsk.TYPE_F16
    act = {"none": bsk.ACT_NONE, "relu": bsk.ACT_RELU, "gelu": bsk.ACT_GELU, "gelu_tanh": bsk.ACT_GELU_TANH, "silu": bsk.ACT_SILU}[c["act"]]
    n, m, k, w, b, kept = c["n"], c["M"], c["K"], st["w"], st["b"], st["kept"]
    if c["op"] == "linear":
        bsk.linear_act_enqueue(kind, w[0], k, st["x"], st["x_stride"], b[0], st["r"], m, st["out"], m, kept[0], m, m, k, n, act)
        return [st["out"]] + (kept if c["keep"] else [])
    if c["op"] == "gated":
        bsk.gated_linear_enqueue(kind, w[0], w[1], k, st["x"], st["x_stride"], b[0], b[1], st["out"], m, kept[0], kept[1], m, m, k, n, act)
        return [st["out"]] + (kept if c["keep"] else [])
    gt = bsk.GRAD_F32 if c["grad32"] else bsk.GRAD_16
    if c["op"] == "linear_backward":
        bsk.linear_act_backward_enqueue(kind, w[0], k, st["x"], st["x_stride"], kept[0], m, st["dy"], m, st["dx"], k, st["dw"][0], k,
                                        st["db"][0], gt, 0, m, k, n, act)
    else:
        bsk.gated_linear_backward_enqueue(kind, w[0], w[1], k, st["x"], st["x_stride"], kept[0], kept[1], m, st["dy"], m, st["dx"], k,
                                          st["dw"][0], st["dw"][1], k, st["db"][0], st["db"][1], gt, 0, m, k, n, act)
    return [st["dx"]] + st["dw"] + (st["db"] if c["bias"] else [])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c = case
    n, m, k = c["n"], c["M"], c["K"]
    parts = 2 if "gated" in c["op"] else 1
    if c["op"] in ("linear", "gated"):
        values = parts * m * k + n * k + n * m + parts * (m * c["bias"] + n * m * c["keep"]) + n * m * c["residual"]
        return {"bytes": 2 * values, "flops": 2 * parts * n * m * k}
    size = 4 if c["grad32"] else 2
    kept = 0 if c["act"] == "none" and parts == 1 else parts
    return {"bytes": 2 * (parts * m * k + n * k + n * m * (1 + kept) + n * k) + size * parts * (m * k + m * c["bias"]),
            "flops": 4 * parts * n * m * k}


def _wide_act(name, z):
    """act(z) and act'(z) in 64 bits, by forms that lose nothing where the values are small."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if name == "gelu":
        p = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * p, p + z * torch.exp(-z * z / 2) * (1 / math.sqrt(2 * math.pi))
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    v = 2 * ROOT_2_OVER_PI * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(v)
    return z * s, s + z * s * torch.sigmoid(-v) * (2 * ROOT_2_OVER_PI) * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    c = case
    if work(c)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    x, w = st["x"].double(), [a.double() for a in st["w"]]
    if c["op"] in ("linear", "gated"):
        z = [torch.mm(x, a.t()) for a in w]
        if c["bias"]:
            z = [a + b.double() for a, b in zip(z, st["b"])]
        y = _wide_act(c["act"], z[0])[0]
        if c["op"] == "gated":
            y = y * z[1]
        if c["residual"]:
            y = y + st["r"].double()
        return [y] + (z if c["keep"] else [])
    a, slope = _wide_act(c["act"], st["kept"][0].double())
    dy = st["dy"].double()
    dz = [dy * st["kept"][1].double() * slope, dy * a] if c["op"] == "gated_backward" else [dy * slope]
    dx = torch.mm(dz[0], w[0])
    if len(dz) > 1:
        dx += torch.mm(dz[1], w[1])
    return [dx] + [torch.mm(d.t(), x) for d in dz] + ([d.sum(0) for d in dz] if c["bias"] else [])
