"""Timing cases of the fused linear and gated feed-forward operators over nested 4-bit weights.

Four operators on a frozen weight W that is held as packed 4-bit codes with nested block scales:

    linear            z = x W^T + bias,  y = act(z) + residual
    linear_backward   dz = dy act'(z),   dx = dz W,   dbias = sum over rows of dz
    gated             h = act(x Wg^T) * (x Wu^T)
    gated_backward    dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu

A weight element is what the dequantization writes for x's type:
W_i = cvt(fl32(codebook4[nibble_i] * fl32(fl32(scale_codebook[code_b] * absmax_{b/256}) + offset))),
b = i / blocksize, cvt the rounding to FP16 or BF16.  It does not depend on the number of tokens.
z, g and u are the pre-activations; where a case saves them they are outputs of the forward pass (a training
step keeps them), and the backward passes take them as inputs.

`own` False: the operators in elementary torch operations, in 32 bits.  `own` True: the framework's calls.
"""
import math

import torch

own = False

#: 4096 x 4096 and 4096 x 11008 / 11008 x 4096 are the square and the mid-size matrix pair of the framework's
#: own workloads, 28672 x 8192 its headline matrix, 1000 x 2376 the ragged shape of its linear tests.
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LARGEST_FLOPS = 4.0 * 4096 * 11008 * 4096
LARGEST_WEIGHT = 28672 * 8192
GELU_C = math.sqrt(2.0 / math.pi)


def _case(name, op, m, n_out, n_in, dtype="bf16", act="none", bias=False, residual=False, save=False,
          blocksize=64):
    return {"name": name, "op": op, "m": m, "n_out": n_out, "n_in": n_in, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "save": save, "blocksize": blocksize}


def listed():
    return [
        # one generated token: attention's output projection, added to the residual stream
        _case("linear_token_4096x4096", "linear", 1, 4096, 4096, residual=True),
        # 16 sequences decoded together: the down projection of a large model's feed-forward block
        _case("linear_batch16_8192x28672", "linear", 16, 8192, 28672, residual=True),
        # a prompt of 2048 tokens: the down projection of a mid-size model's feed-forward block
        _case("linear_prompt2048_4096x11008", "linear", 2048, 4096, 11008, residual=True),
        # a plain (ungated) feed-forward layer in FP16 with a bias, ragged sizes, kept for training
        _case("linear_ragged37_1000x2376", "linear", 37, 1000, 2376, dtype="f16", act="gelu", bias=True,
              save=True),
        # its gradient at a training micro-batch of 512 tokens
        _case("linear_backward512_11008x4096", "linear_backward", 512, 11008, 4096, act="gelu", bias=True),
        # an odd head: every row starts in the middle of a byte and of a block
        _case("linear_backward_odd150_1001x1377", "linear_backward", 150, 1001, 1377, dtype="f16",
              act="gelu_tanh", bias=True, blocksize=128),
        # one generated token through the gated half of a large model's feed-forward block
        _case("gated_token_28672x8192", "gated", 1, 28672, 8192, act="silu"),
        # 64 sequences decoded together, mid-size model, FP16
        _case("gated_batch64_11008x4096", "gated", 64, 11008, 4096, dtype="f16", act="silu"),
        # a training micro-batch of 512 tokens of the large model: the pre-activations are kept
        _case("gated_train512_28672x8192", "gated", 512, 28672, 8192, act="silu", save=True),
        # a prompt of 4096 tokens, mid-size model
        _case("gated_prompt4096_11008x4096", "gated", 4096, 11008, 4096, act="silu"),
        # a training step of 2048 tokens, mid-size model
        _case("gated_backward2048_11008x4096", "gated_backward", 2048, 11008, 4096, act="silu"),
        # the last, short micro-batch of a small ragged model
        _case("gated_backward_ragged37_1000x2376", "gated_backward", 37, 1000, 2376, dtype="f16",
              act="gelu_tanh"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "linear_backward", "gated", "gated_backward"])
    gated = op.startswith("gated")
    n_out, n_in = _spread(rng, 64, 28672), _spread(rng, 64, 28672)
    step = rng.choice([1, 1, 8, 64, 64])  # odd widths, and those that models have
    n_out, n_in = max(n_out // step * step, 1), max(n_in // step * step, 1)
    while n_out * n_in > LARGEST_WEIGHT:
        n_out = max(n_out // 2 // step * step, 1)
    most = LARGEST_FLOPS / (2.0 * n_out * n_in * (2 if gated else 1))
    m = min(_spread(rng, 1, 4096), max(int(most), 1))
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] + ([] if gated else ["none"]))
    return {"op": op, "m": m, "n_out": n_out, "n_in": n_in, "dtype": rng.choice(["f16", "bf16"]),
            "act": act, "bias": not gated and rng.random() < 0.5,
            "residual": op == "linear" and rng.random() < 0.5,
            "save": op in ("linear", "gated") and rng.random() < 0.5,
            "blocksize": rng.choice([32, 64, 64, 128, 256, 1024, 4096])}


# ----------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------
def _make_weight(gen, n, blocksize):
    """Uniform codes, lognormal nested maxima, a sorted scale codebook and a sorted 16-value codebook with an
    exact zero; the offset is the size of the mean block scale, as the nested quantization leaves it."""
    dev = gen.device
    blocks = -(-n // blocksize)
    groups = -(-blocks // 256)
    cb4 = torch.rand(15, generator=gen, device=dev) * 2 - 1
    return {
        "packed": torch.randint(0, 256, (-(-n // 2),), generator=gen, device=dev, dtype=torch.uint8),
        "scale_codes": torch.randint(0, 256, (blocks,), generator=gen, device=dev, dtype=torch.uint8),
        "nested_absmax": torch.exp(torch.randn(groups, generator=gen, device=dev) * 0.5 - 3.0),
        "scale_codebook": torch.sort(torch.rand(256, generator=gen, device=dev) * 2 - 1).values,
        "codebook4": torch.sort(torch.cat([cb4, torch.zeros(1, device=dev)])).values,
        "offset": 0.03,
    }


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    m, n_out, n_in, dt = case["m"], case["n_out"], case["n_in"], TYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    s = dict(case)
    gated = case["op"].startswith("gated")
    s["weights"] = [_make_weight(gen, n_out * n_in, case["blocksize"]) for _ in range(2 if gated else 1)]
    if case["op"].endswith("backward"):
        s["grad"] = normal(m, n_out, scale=0.5)
        if gated:
            s["gate_pre"], s["up_pre"] = normal(m, n_out, scale=1.5), normal(m, n_out, scale=1.5)
        elif case["act"] != "none":
            s["pre"] = normal(m, n_out, scale=1.5)
    else:
        s["x"] = normal(m, n_in)
        if case["bias"]:
            s["bias_v"] = normal(n_out, scale=0.2)
        if case["residual"]:
            s["residual_v"] = normal(m, n_out)
    return s


# ----------------------------------------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------------------------------------
def _weight(w, n_out, n_in, blocksize, dt):
    n = n_out * n_in
    blocks = w["scale_codes"].numel()
    scale = w["scale_codebook"][w["scale_codes"].long()]
    scale = scale * w["nested_absmax"].repeat_interleave(256)[:blocks]
    scale = scale + w["offset"]
    nibbles = torch.stack((w["packed"] & 15, w["packed"] >> 4), 1).reshape(-1)[:n]
    values = w["codebook4"][nibbles.int()]
    values = torch.nn.functional.pad(values, (0, blocks * blocksize - n)).view(blocks, blocksize)
    values = (values * scale[:, None]).reshape(-1)[:n]
    return values.to(dt).float().view(n_out, n_in)


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    return z / (1 + torch.exp(-2 * GELU_C * (z + 0.044715 * z * z * z)))


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s = 1 / (1 + torch.exp(-2 * GELU_C * (z + 0.044715 * z * z * z)))
    return s + z * s * (1 - s) * 2 * GELU_C * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    n_out, n_in, dt, act = s["n_out"], s["n_in"], TYPES[s["dtype"]], s["act"]
    ws = [_weight(w, n_out, n_in, s["blocksize"], dt) for w in s["weights"]]
    if s["op"] == "linear":
        z = s["x"].float() @ ws[0].t()
        if s["bias"]:
            z = z + s["bias_v"].float()
        y = _act(act, z)
        if s["residual"]:
            y = y + s["residual_v"].float()
        return {"y": y.to(dt), "pre": z.to(dt) if s["save"] else None}
    if s["op"] == "linear_backward":
        dz = s["grad"].float()
        if act != "none":
            dz = dz * _act_grad(act, s["pre"].float())
        return {"dx": (dz @ ws[0]).to(dt), "dz": dz.to(dt), "dbias": dz.sum(0) if s["bias"] else None}
    if s["op"] == "gated":
        x = s["x"].float()
        g, u = x @ ws[0].t(), x @ ws[1].t()
        h = _act(act, g) * u
        return {"h": h.to(dt), "gate_pre": g.to(dt) if s["save"] else None, "up_pre": u.to(dt) if s["save"] else None}
    dh, g, u = s["grad"].float(), s["gate_pre"].float(), s["up_pre"].float()
    dg, du = dh * u * _act_grad(act, g), dh * _act(act, g)
    return {"dx": (dg @ ws[0] + du @ ws[1]).to(dt), "dgate": dg.to(dt), "dup": du.to(dt)}


# ----------------------------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------------------------
def _own(s):
    import block_wise_bit_amd as dq4

    sizes = (s["n_out"], s["n_in"], s["blocksize"])
    if s["op"] == "linear":
        pre = s["x"].new_empty((s["m"], s["n_out"])) if s["save"] else None
        y = dq4.dq4_linear_fused(**s["weights"][0], n_out=sizes[0], n_in=sizes[1], blocksize=sizes[2], x=s["x"],
                                 bias=s.get("bias_v"), residual=s.get("residual_v"), activation=s["act"], pre=pre)
        return {"y": y, "pre": pre}
    if s["op"] == "linear_backward":
        dx, dz, dbias = dq4.dq4_linear_fused_backward(
            **s["weights"][0], n_out=sizes[0], n_in=sizes[1], blocksize=sizes[2], dy=s["grad"], pre=s.get("pre"),
            activation=s["act"], bias_grad=s["bias"])
        return {"dx": dx, "dz": dz, "dbias": dbias}
    if s["op"] == "gated":
        g, u = (s["x"].new_empty((2, s["m"], s["n_out"])) if s["save"] else (None, None))
        h = dq4.dq4_gated_fused(s["weights"][0], s["weights"][1], *sizes, x=s["x"], activation=s["act"], gate_pre=g,
                                up_pre=u)
        return {"h": h, "gate_pre": g, "up_pre": u}
    dx, dgate, dup = dq4.dq4_gated_fused_backward(
        s["weights"][0], s["weights"][1], *sizes, dh=s["grad"], gate_pre=s["gate_pre"], up_pre=s["up_pre"],
        activation=s["act"])
    return {"dx": dx, "dgate": dgate, "dup": dup}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    m, n_out, n_in, n = case["m"], case["n_out"], case["n_in"], case["n_out"] * case["n_in"]
    gated = case["op"].startswith("gated")
    blocks = -(-n // case["blocksize"])
    weight = -(-n // 2) + blocks + 4 * -(-blocks // 256) + 4 * (256 + 16)
    wide, narrow = 2.0 * m * n_out, 2.0 * m * n_in  # bytes of an m x n_out and an m x n_in matrix
    if case["op"] == "linear":
        moved = narrow + wide * (1 + case["residual"] + case["save"]) + 2.0 * n_out * case["bias"]
    elif case["op"] == "linear_backward":
        moved = narrow + wide * (1 if case["act"] == "none" else 3) + 4.0 * n_out * case["bias"]
    elif case["op"] == "gated":
        moved = narrow + wide * (1 + 2 * case["save"])
    else:
        moved = narrow + wide * 5
    return {"bytes": weight * (2 if gated else 1) + moved, "flops": 2.0 * m * n * (2 if gated else 1)}


# ----------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    m, n_out, n_in, dt, bs = case["m"], case["n_out"], case["n_in"], TYPES[case["dtype"]], case["blocksize"]

    def wide(t):
        return t.to(torch.float64)

    def single(t):  # one rounding to binary32; the products and sums below are exact in 64 bits before it
        return wide(t.to(torch.float32))

    def matrix(w):
        i = torch.arange(n_out * n_in, device="cuda")
        b = torch.arange(w["scale_codes"].numel(), device="cuda")
        offset = float(torch.tensor(w["offset"], dtype=torch.float32))
        t = single(wide(w["scale_codebook"]).take(w["scale_codes"].to(torch.int64)) * wide(w["nested_absmax"]).take(b // 256))
        scale = single(t + offset)
        byte = w["packed"].take(i // 2).to(torch.int32)
        code = torch.where(i % 2 == 0, byte % 16, byte // 16).to(torch.int64)
        v = wide(w["codebook4"]).take(code)
        del byte, code
        v *= scale.take(i // bs)
        return wide(v.to(torch.float32).to(dt)).reshape(n_out, n_in)

    def phi(z):  # the normal distribution's integral
        return torch.special.ndtr(z)

    def value(z):
        return {"none": lambda: z, "relu": lambda: torch.clamp(z, min=0.0), "silu": lambda: z * torch.sigmoid(z),
                "gelu": lambda: z * phi(z),
                "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z ** 3)))}[case["act"]]()

    def slope(z):
        def tanh_form():
            t = torch.tanh(GELU_C * (z + 0.044715 * z ** 3))
            return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 0.134145 * z ** 2)
        return {"none": lambda: torch.ones_like(z), "relu": lambda: torch.heaviside(z, torch.zeros_like(z)),
                "silu": lambda: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z),
                "gelu": lambda: phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                "gelu_tanh": tanh_form}[case["act"]]()

    if case["op"] == "linear":
        z = torch.matmul(wide(s["x"]), matrix(s["weights"][0]).T)
        z = z + wide(s["bias_v"]) if case["bias"] else z
        y = value(z) + wide(s["residual_v"]) if case["residual"] else value(z)
        return {"y": y, "pre": z if case["save"] else None}
    if case["op"] == "linear_backward":
        dz = wide(s["grad"]) * (slope(wide(s["pre"])) if case["act"] != "none" else 1.0)
        dx = torch.matmul(dz, matrix(s["weights"][0]))
        return {"dx": dx, "dz": dz, "dbias": torch.sum(dz, dim=0) if case["bias"] else None}
    if case["op"] == "gated":
        g = torch.matmul(wide(s["x"]), matrix(s["weights"][0]).T)
        u = torch.matmul(wide(s["x"]), matrix(s["weights"][1]).T)
        keep = case["save"]
        return {"h": value(g) * u, "gate_pre": g if keep else None, "up_pre": u if keep else None}
    dh, g, u = wide(s["grad"]), wide(s["gate_pre"]), wide(s["up_pre"])
    dgate, dup = dh * u * slope(g), dh * value(g)
    dx = torch.matmul(dgate, matrix(s["weights"][0])) + torch.matmul(dup, matrix(s["weights"][1]))
    return {"dx": dx, "dgate": dgate, "dup": dup}
