"""Timing cases of the LLM.int8 linear layer and of a mixture-of-experts layer over nested 4-bit weights.

Four paths, T the 16-bit type of a case (FP16 or BF16):

    int8_quant     each token's row x_i to 8-bit codes: s_i = max |x_ij| over its elements below the threshold,
                   code = round(127 x / s), half to even; the columns in which an element reaches the threshold
                   ("outliers") are listed, in ascending order, and their codes are 0
    int8_linear    y = (codes CB^T) s_i S_n / 127^2 + x[:, outliers] Wt[:, outliers]^T + bias + residual, with the
                   weight's 8-bit codes CB, its row scales S and Wt = T(fl32(fl32(CB S) / 127))
    int8_backward  dx = dy Wt, dbias = sum over rows of dy
    moe            router logits x R^T, the top_k experts of each token and their softmax weights w, then
                   y = sum over the chosen experts e of w_e (act(x Wg_e^T) * (x Wu_e^T)) Wd_e^T + residual

A 4-bit weight's element is what the dequantization writes for T:
W_i = cvt(fl32(codebook4[nibble_i] * fl32(fl32(scale_codebook[code_b] * absmax_{b/256}) + offset))), b = i / blocksize.
The experts' matrices are stacked by rows: one weight of (experts n_ff) x n_in for Wg and for Wu, one of
(experts n_in) x n_ff for Wd.

`own` False: the operators in elementary torch operations, in 32 bits (64 where a code or the choice of an expert
lies next to a border).  `own` True: the framework's calls.
"""
import math

import torch

own = False

#: 4096 x 4096, 4096 x 11008 / 11008 x 4096 and 4096 x 14336 are matrices of the framework's own workloads, 28672 x
#: 8192 its headline matrix, 1000 x 2376 the ragged shape of its linear tests.  6.0 is LLM.int8's threshold.
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
THRESHOLD = 6.0
LARGEST_FLOPS = 2.0 * 4096 * 11008 * 4096
LARGEST_WEIGHT = 28672 * 8192
LARGEST_TOKENS = 4096 * 4096      # elements of an x that is quantized
LARGEST_EXPERTS = 8 * 14336 * 4096  # elements of one stacked matrix
GELU_C = math.sqrt(2.0 / math.pi)


def _quant(name, m, n_in, dtype="f16", threshold=THRESHOLD, outliers=0):
    return {"name": name, "op": "int8_quant", "m": m, "n_in": n_in, "dtype": dtype, "threshold": threshold,
            "outliers": outliers}


def _linear(name, m, n_out, n_in, dtype="f16", outliers=0, bias=False, residual=False):
    return {"name": name, "op": "int8_linear", "m": m, "n_out": n_out, "n_in": n_in, "dtype": dtype,
            "outliers": outliers, "bias": bias, "residual": residual}


def _backward(name, m, n_out, n_in, dtype="bf16", bias=False):
    return {"name": name, "op": "int8_backward", "m": m, "n_out": n_out, "n_in": n_in, "dtype": dtype, "bias": bias}


def _moe(name, m, experts, top_k, n_ff, n_in, dtype="bf16", act="silu", blocksize=64, residual=True, renormalize=True):
    return {"name": name, "op": "moe", "m": m, "experts": experts, "top_k": top_k, "n_ff": n_ff, "n_in": n_in,
            "dtype": dtype, "act": act, "blocksize": blocksize, "residual": residual, "renormalize": renormalize}


def listed():
    return [
        # one generated token before a wide layer; a few of its channels are outliers
        _quant("int8_quant_token_8192", 1, 8192, outliers=5),
        # a prompt of 4096 tokens
        _quant("int8_quant_prompt4096_4096", 4096, 4096, outliers=24),
        # one generated token: attention's output projection, added to the residual stream
        _linear("int8_linear_token_4096x4096", 1, 4096, 4096, outliers=3, residual=True),
        # 16 sequences decoded together: a feed-forward layer with a bias
        _linear("int8_linear_batch16_14336x4096", 16, 14336, 4096, outliers=16, bias=True),
        # the last, short part of a prompt in a ragged model: no row starts on a 16-byte boundary
        _linear("int8_linear_odd150_1001x1377", 150, 1001, 1377, dtype="bf16", residual=True),
        # a prompt of 2048 tokens through a down projection, with many outlier channels
        _linear("int8_linear_prompt2048_4096x14336", 2048, 4096, 14336, outliers=64, residual=True),
        # a prompt of 4096 tokens without any
        _linear("int8_linear_prompt4096_11008x4096", 4096, 11008, 4096, dtype="bf16"),
        # a training micro-batch of 512 tokens
        _backward("int8_backward512_11008x4096", 512, 11008, 4096, bias=True),
        # the short micro-batch of a small ragged model
        _backward("int8_backward_ragged37_1000x2376", 37, 1000, 2376, dtype="f16", bias=True),
        # one generated token, many small experts
        _moe("moe_token_64x1024x2048", 1, 64, 8, 1024, 2048),
        # 16 sequences decoded together, few large experts
        _moe("moe_batch16_8x14336x4096", 16, 8, 2, 14336, 4096, dtype="f16"),
        # 64 sequences, a ragged model, weights of the softmax over all experts
        _moe("moe_batch64_16x1000x2376", 64, 16, 4, 1000, 2376, act="gelu_tanh", blocksize=128, residual=False,
             renormalize=False),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _stepped(rng, low, high):
    step = rng.choice([1, 1, 8, 64, 64])  # odd widths, and those that models have
    return max(_spread(rng, low, high) // step * step, 1)


def draw(rng):
    op = rng.choice(["int8_quant", "int8_linear", "int8_linear", "int8_backward", "moe", "moe"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "int8_quant":
        n_in = _stepped(rng, 64, 28672)
        m = min(_spread(rng, 1, 4096), LARGEST_TOKENS // n_in)
        return {"op": op, "m": m, "n_in": n_in, "dtype": dtype, "threshold": rng.choice([0.0, THRESHOLD]),
                "outliers": min(rng.randrange(65), n_in)}
    if op == "moe":
        experts = _spread(rng, 4, 128)
        n_ff, n_in = _stepped(rng, 64, 14336), _stepped(rng, 64, 8192)
        while experts * n_ff * n_in > LARGEST_EXPERTS:
            n_ff = max(n_ff // 2, 1)
        return {"op": op, "m": _spread(rng, 1, 64), "experts": experts, "top_k": rng.randint(1, min(experts, 8)),
                "n_ff": n_ff, "n_in": n_in, "dtype": dtype, "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                "blocksize": rng.choice([32, 64, 64, 128, 256, 1024, 4096]), "residual": rng.random() < 0.5,
                "renormalize": rng.random() < 0.7}
    n_out, n_in = _stepped(rng, 64, 28672), _stepped(rng, 64, 28672)
    while n_out * n_in > LARGEST_WEIGHT:
        n_out = max(n_out // 2, 1)
    m = min(_spread(rng, 1, 4096), max(int(LARGEST_FLOPS / (2.0 * n_out * n_in * (2 if op == "int8_backward" else 1))), 1))
    case = {"op": op, "m": m, "n_out": n_out, "n_in": n_in, "dtype": dtype, "bias": rng.random() < 0.5}
    if op == "int8_linear":
        case.update(outliers=rng.choice([0, rng.randrange(1, 65)]), residual=rng.random() < 0.5)
    return case


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
    gen.manual_seed(int(seed) * 1000003 + 29)
    m, n_in, dt = case["m"], case["n_in"], TYPES[case["dtype"]]
    s = dict(case)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    def tokens(outliers):
        """Hidden states: a normal bulk that stays below the threshold, and some channels far above it."""
        x = torch.randn(m, n_in, generator=gen, device="cuda").clamp_(-5.5, 5.5)
        cols = torch.sort(torch.randperm(n_in, generator=gen, device="cuda")[:outliers]).values
        x[:, cols] = x[:, cols] * 4.0 + torch.where(x[:, cols] < 0, -8.0, 8.0)
        return x.to(dt), cols

    if case["op"] == "int8_quant":
        s["x"] = tokens(case["outliers"])[0]
    elif case["op"] == "moe":
        n_ff, experts = case["n_ff"], case["experts"]
        s["x"] = normal(m, n_in)
        s["router"] = normal(experts, n_in, scale=1.0 / math.sqrt(n_in))
        s["gate"], s["up"], s["down"] = (_make_weight(gen, experts * n_ff * n_in, case["blocksize"]) for _ in range(3))
        s["residual_v"] = normal(m, n_in) if case["residual"] else None
    else:
        n_out = case["n_out"]
        s["CB"] = torch.randint(-127, 128, (n_out, n_in), generator=gen, device="cuda", dtype=torch.int8)
        s["SCB"] = torch.rand(n_out, generator=gen, device="cuda") * 0.08 + 0.02
        if case["op"] == "int8_backward":
            s["dy"] = normal(m, n_out, scale=0.5)
        else:
            s["x"], cols = tokens(case["outliers"])
            small = s["x"].float()
            small[:, cols] = 0
            s["scales"] = small.abs().amax(1)
            s["codes"] = torch.round(small * (127.0 / s["scales"].clamp(min=1e-30))[:, None]).to(torch.int8)
            s["outlier_list"] = None
            if case["outliers"]:
                s["outlier_list"] = torch.full((1 + n_in,), -1, dtype=torch.int32, device="cuda")
                s["outlier_list"][0] = len(cols)
                s["outlier_list"][1:1 + len(cols)] = cols
            s["bias_v"] = normal(n_out, scale=0.2) if case["bias"] else None
            s["residual_v"] = normal(m, n_out) if case["residual"] else None
    return s


# ----------------------------------------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------------------------------------
def _weight(w, rows, cols, blocksize, dt):
    n = rows * cols
    blocks = w["scale_codes"].numel()
    scale = w["scale_codebook"][w["scale_codes"].long()]
    scale = scale * w["nested_absmax"].repeat_interleave(256)[:blocks]
    scale = scale + w["offset"]
    nibbles = torch.stack((w["packed"] & 15, w["packed"] >> 4), 1).reshape(-1)[:n]
    values = w["codebook4"][nibbles.int()]
    values = torch.nn.functional.pad(values, (0, blocks * blocksize - n)).view(blocks, blocksize)
    values = (values * scale[:, None]).reshape(-1)[:n]
    return values.to(dt).float().view(rows, cols)


def _experts(w, ids, rows, cols, blocksize, dt):
    """The rows x cols matrices of the experts `ids`, element by element out of the stacked weight."""
    n = rows * cols
    i = (ids[:, None] * n + torch.arange(n, device=ids.device)).view(-1)
    block = i // blocksize
    scale = w["scale_codebook"][w["scale_codes"][block].int()] * w["nested_absmax"][block // 256] + w["offset"]
    nibbles = (w["packed"][i // 2].int() >> (4 * (i % 2))) & 15
    return (w["codebook4"][nibbles] * scale).to(dt).float().view(-1, rows, cols)


def _act(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    return z / (1 + torch.exp(-2 * GELU_C * (z + 0.044715 * z * z * z)))


def _values(codes, scales):
    """What 8-bit codes stand for."""
    return codes * (scales * (1.0 / 127.0))[:, None]


def _plain_quant(s):
    x = s["x"].double()
    big = (~(x.abs() < s["threshold"])) if s["threshold"] > 0 else torch.zeros_like(x, dtype=torch.bool)
    scales = torch.where(big, 0.0, x).abs().amax(1)
    column = big.any(0)
    codes = torch.where(column | (scales == 0)[:, None], 0.0, torch.round(127.0 * x / scales[:, None]))
    outliers = None
    if s["threshold"] > 0:
        k = x.shape[1]
        order = torch.sort(torch.where(column, torch.arange(k, device=x.device), k)).values
        outliers = torch.cat((column.sum().view(1), torch.where(order < k, order, -1))).int()
    scales = scales.float()
    return {"values": _values(codes.float(), scales), "scales": scales, "outliers": outliers}


def _plain_linear(s):
    dt = TYPES[s["dtype"]]
    y = (s["codes"].float() @ s["CB"].float().t()) * (s["scales"][:, None] * s["SCB"] / 16129.0)
    if s["outlier_list"] is not None:
        cols = s["outlier_list"][1:1 + s["outliers"]].long()
        wt = (s["CB"][:, cols].float() * s["SCB"][:, None] * (1.0 / 127.0)).to(dt).float()
        y = y + s["x"][:, cols].float() @ wt.t()
    if s["bias"]:
        y = y + s["bias_v"].float()
    if s["residual"]:
        y = y + s["residual_v"].float()
    return {"y": y.to(dt)}


def _plain_backward(s):
    dt = TYPES[s["dtype"]]
    wt = (s["CB"].float() * s["SCB"][:, None] * (1.0 / 127.0)).to(dt).float()
    dy = s["dy"].float()
    return {"dx": (dy @ wt).to(dt), "dbias": dy.sum(0) if s["bias"] else None}


def _plain_moe(s):
    m, experts, n_ff, n_in, dt = s["m"], s["experts"], s["n_ff"], s["n_in"], TYPES[s["dtype"]]
    logits = s["x"].double() @ s["router"].double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: the lowest index first
    ids, top = order.indices[:, :s["top_k"]], order.values[:, :s["top_k"]]
    shift = top[:, :1]
    weights = torch.exp(top - shift)
    weights = weights / (weights if s["renormalize"] else torch.exp(logits - shift)).sum(1, keepdim=True)
    x = s["x"].float()
    if m * s["top_k"] < experts:  # fewer choices than experts: the chosen matrices, one for each choice
        chosen, xs = ids.reshape(-1), x.repeat_interleave(s["top_k"], 0)[:, :, None]
        g = _experts(s["gate"], chosen, n_ff, n_in, s["blocksize"], dt) @ xs
        u = _experts(s["up"], chosen, n_ff, n_in, s["blocksize"], dt) @ xs
        out = _experts(s["down"], chosen, n_in, n_ff, s["blocksize"], dt) @ (_act(s["act"], g) * u)
        y = (out.view(m, s["top_k"], n_in) * weights.float()[:, :, None]).sum(1)
        return _plain_moe_end(s, y, ids, weights)
    # every expert on every token, and the weights of those that were chosen
    share = torch.zeros_like(logits).scatter_(1, ids, weights).float()
    g = x @ _weight(s["gate"], experts * n_ff, n_in, s["blocksize"], dt).t()
    u = x @ _weight(s["up"], experts * n_ff, n_in, s["blocksize"], dt).t()
    h = (_act(s["act"], g) * u).view(m, experts, n_ff).transpose(0, 1)
    down = _weight(s["down"], experts * n_in, n_ff, s["blocksize"], dt).view(experts, n_in, n_ff)
    y = (torch.matmul(down, h.transpose(1, 2).contiguous()) * share.t()[:, None, :]).sum(0).t()
    return _plain_moe_end(s, y, ids, weights)


def _plain_moe_end(s, y, ids, weights):
    if s["residual"]:
        y = y + s["residual_v"].float()
    return {"y": y.to(TYPES[s["dtype"]]), "ids": ids.int(), "weights": weights.float()}


# ----------------------------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------------------------
def _own(s):
    import block_wise_bit_amd as dq4

    if s["op"] == "int8_quant":
        codes, scales, outliers = dq4.dq4_int8_quant(s["x"], threshold=s["threshold"])
        return {"values": _values(codes, scales), "scales": scales, "outliers": outliers}
    if s["op"] == "int8_linear":
        mixed = {} if s["outlier_list"] is None else {"x": s["x"], "outliers": s["outlier_list"]}
        return {"y": dq4.dq4_int8_linear(s["codes"], s["scales"], s["CB"], s["SCB"], dtype=TYPES[s["dtype"]],
                                         bias=s["bias_v"], residual=s["residual_v"], **mixed)}
    if s["op"] == "int8_backward":
        dx, dbias = dq4.dq4_int8_linear_backward(s["dy"], s["CB"], s["SCB"], bias_grad=s["bias"])
        return {"dx": dx, "dbias": dbias}
    ids, weights = dq4.dq4_moe_route(s["x"], s["router"], s["top_k"], renormalize=s["renormalize"])
    y = dq4.dq4_moe_fused(s["gate"], s["up"], s["down"], s["experts"], s["n_ff"], s["n_in"], s["blocksize"], s["x"],
                          ids, weights, activation=s["act"], residual=s["residual_v"])
    return {"y": y, "ids": ids, "weights": weights}


def run(state):
    if own:
        return _own(state)
    return {"int8_quant": _plain_quant, "int8_linear": _plain_linear, "int8_backward": _plain_backward,
            "moe": _plain_moe}[state["op"]](state)


def work(case):
    m, k = case["m"], case["n_in"]
    if case["op"] == "int8_quant":
        # the codes are returned as FP32 values: 2 bytes read and 4 written for each
        return {"bytes": 6.0 * m * k + 4.0 * m + 4.0 * (1 + k), "flops": 4.0 * m * k}
    if case["op"] == "moe":
        experts, n_ff, top_k = case["experts"], case["n_ff"], case["top_k"]
        # the experts that some token is expected to choose, all experts being alike
        used = experts * (1.0 - (1.0 - top_k / experts) ** m)
        n = n_ff * k
        matrix = n / 2 + n / case["blocksize"] + n / case["blocksize"] / 64
        rows = 2.0 * m * k
        return {"bytes": 3 * used * matrix + rows * (2 + case["residual"]) + 2.0 * experts * k + 8.0 * m * top_k,
                "flops": 2.0 * m * experts * k + 6.0 * m * top_k * n}
    n = case["n_out"]
    if case["op"] == "int8_backward":
        return {"bytes": 1.0 * n * k + 4.0 * n + 2.0 * m * (n + k) + 4.0 * n * case["bias"], "flops": 2.0 * m * n * k}
    moved = 1.0 * (m + n) * k + 4.0 * (m + n) + 2.0 * m * n * (1 + case["residual"]) + 2.0 * n * case["bias"]
    outliers = case["outliers"]
    return {"bytes": moved + 2.0 * m * outliers + 4.0 * outliers, "flops": 2.0 * m * n * (k + outliers)}


# ----------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    dt = TYPES[case["dtype"]]

    def wide(t):
        return t.to(torch.float64)

    def single(t):  # one rounding to binary32; the products and sums below are exact in 64 bits before it
        return wide(t.to(torch.float32))

    def int8_weight(rows_scale, codes):
        r127 = float(torch.tensor(1.0 / 127.0, dtype=torch.float32))
        return wide(single(single(wide(codes) * wide(rows_scale).unsqueeze(1)) * r127).to(torch.float32).to(dt))

    if case["op"] == "int8_quant":
        x = wide(s["x"])
        small = torch.abs(x) < case["threshold"] if case["threshold"] > 0 else torch.ones_like(x, dtype=torch.bool)
        peak = torch.max(torch.abs(x) * small, dim=1, keepdim=True).values
        kept = torch.all(small, dim=0, keepdim=True)
        # 127 x / s is a quotient of short integers: rounded to 64 bits it is on a half only if it is one
        codes = torch.round(x * 127.0 / torch.clamp(peak, min=1e-300)) * kept
        listed_columns = torch.nonzero(~kept[0]).flatten()
        outliers = None
        if case["threshold"] > 0:
            outliers = torch.full((1 + case["n_in"],), -1, dtype=torch.int32, device="cuda")
            outliers[0] = listed_columns.numel()
            outliers[1:1 + listed_columns.numel()] = listed_columns.to(torch.int32)
        return {"values": codes * peak / 127.0, "scales": peak.flatten(), "outliers": outliers}
    if case["op"] == "int8_linear":
        # sums of products of 8-bit integers: whole numbers below 2^53
        sums = torch.matmul(wide(s["codes"]), wide(s["CB"]).T)
        y = sums * wide(s["scales"]).unsqueeze(1) * wide(s["SCB"]).unsqueeze(0) / (127.0 * 127.0)
        if case["outliers"]:
            cols = s["outlier_list"][1:1 + case["outliers"]].to(torch.int64)
            wt = int8_weight(s["SCB"], s["CB"].index_select(1, cols))
            y = y + torch.matmul(wide(s["x"].index_select(1, cols)), wt.T)
        y = y + wide(s["bias_v"]) if case["bias"] else y
        return {"y": y + wide(s["residual_v"]) if case["residual"] else y}
    if case["op"] == "int8_backward":
        dx = torch.matmul(wide(s["dy"]), int8_weight(s["SCB"], s["CB"]))
        return {"dx": dx, "dbias": torch.sum(wide(s["dy"]), dim=0) if case["bias"] else None}

    m, experts, top_k, n_ff, n_in = case["m"], case["experts"], case["top_k"], case["n_ff"], case["n_in"]

    def expert_rows(w, first, rows, cols):
        """Rows first .. first + rows - 1 of a stacked weight."""
        i = torch.arange(first * cols, (first + rows) * cols, device="cuda")
        b = torch.div(i, case["blocksize"], rounding_mode="floor")
        offset = float(torch.tensor(w["offset"], dtype=torch.float32))
        t = single(wide(w["scale_codebook"]).take(w["scale_codes"].take(b).to(torch.int64))
                   * wide(w["nested_absmax"]).take(torch.div(b, 256, rounding_mode="floor")))
        byte = w["packed"].take(torch.div(i, 2, rounding_mode="floor")).to(torch.int32)
        code = torch.where(i % 2 == 0, byte % 16, torch.div(byte, 16, rounding_mode="floor")).to(torch.int64)
        v = wide(w["codebook4"]).take(code) * single(t + offset)
        return wide(v.to(torch.float32).to(dt)).reshape(rows, cols)

    def value(z):
        return {"relu": lambda: torch.clamp(z, min=0.0), "silu": lambda: z * torch.sigmoid(z),
                "gelu": lambda: z * torch.special.ndtr(z),
                "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z ** 3)))}[case["act"]]()

    x = wide(s["x"])
    logits = torch.matmul(x, wide(s["router"]).T)
    # rank of an expert: how many are larger, or as large with a lower index
    before = torch.ones(experts, experts, device="cuda").triu(1).to(torch.bool)  # [other, this]: other < this
    over = (logits.unsqueeze(2) > logits.unsqueeze(1)) | ((logits.unsqueeze(2) == logits.unsqueeze(1)) & before)
    rank = over.sum(1)
    chosen = rank < top_k
    share = torch.softmax(logits, dim=1)
    share = share * chosen
    if case["renormalize"]:
        share = share / share.sum(1, keepdim=True)
    ids = torch.argsort(rank, dim=1)[:, :top_k]
    y = torch.zeros(m, n_in, dtype=torch.float64, device="cuda")
    for e in range(experts):
        rows = torch.nonzero(chosen[:, e]).flatten()
        if rows.numel() == 0:
            continue
        xe = x.index_select(0, rows)
        g = torch.matmul(xe, expert_rows(s["gate"], e * n_ff, n_ff, n_in).T)
        u = torch.matmul(xe, expert_rows(s["up"], e * n_ff, n_ff, n_in).T)
        out = torch.matmul(value(g) * u, expert_rows(s["down"], e * n_in, n_in, n_ff).T)
        y.index_add_(0, rows, out * share.index_select(0, rows)[:, e:e + 1])
    y = y + wide(s["residual_v"]) if case["residual"] else y
    return {"y": y, "ids": ids.to(torch.int32), "weights": torch.gather(share, 1, ids)}
