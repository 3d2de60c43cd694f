"""Microscaled 4-bit floating point (MXFP4), measured at the sizes a model meets.

* ``quant``: rows coded to E2M1 with one power-of-two scale for each 32 elements, and decoded again;
* ``gemm``: the product of MXFP4 weights with fp16 rows (``a16``), with E4M3 rows of one float32 scale each (``a8``), or
  with fp16 rows that are coded to MXFP4 first (``a4``);
* ``moe``: a whole mixture-of-experts layer on MXFP4 weights for a few tokens, from the router's logits to the layer's output.

``run`` computes the plain form (elementary torch operations in float32, rounded once at the end), or, with ``own`` set,
calls the framework's operators. Codes lie two a byte, the even element in the low four bits; a scale byte s stands for 2^(s - 127).
"""
import math

import torch

own = False

# the largest listed cases: bytes of a coding, operations of a product, bytes of a layer's weights
MOST_CODED, MOST_FLOPS, MOST_WEIGHTS = 11008 * 4096 * 9.1, 2.0 * 2048 * 11008 * 4096, 64 * 3 * 4096 * 1536 * 0.54


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's row before a 4-bit product: only latency counts
        _quant("quant_token", rows=1, K=4096, kind="f16"),
        # a weight matrix, offline
        _quant("quant_weight", rows=11008, K=4096, kind="f32"),
        # one token through an attention projection
        _gemm("gemm_a16_token", acts="a16", M=1, N=4096, K=4096, out="f16", bias=False),
        # a served batch's step through a wide projection, an odd number of sequences
        _gemm("gemm_a16_batch", acts="a16", M=27, N=11008, K=4096, out="f16", bias=False),
        # a chunk of a prompt whose rows stay in fp16
        _gemm("gemm_a16_chunk", acts="a16", M=777, N=4096, K=4096, out="f16", bias=False),
        # ragged decode rows from a norm, the sizes of a 3200-wide model: K ends inside a tile
        _gemm("gemm_a8_ragged", acts="a8", M=45, N=3200, K=8640, out="f16", bias=True),
        # a whole prompt whose rows a norm has coded to E4M3
        _gemm("gemm_a8_prompt", acts="a8", M=2048, N=4096, K=11008, out="f16", bias=False),
        # a small batch on 4-bit rows, float32 sums handed on
        _gemm("gemm_a4_batch", acts="a4", M=8, N=4096, K=11008, out="f32", bias=False),
        # a whole prompt on 4-bit rows
        _gemm("gemm_a4_prompt", acts="a4", M=2048, N=11008, K=4096, out="f16", bias=False),
        # one token through a layer of many small experts
        _moe("moe_token", tokens=1, H=4096, I=1536, experts=64, top=4, act="silu", renorm=True, kind="f32"),
        # a decode step of 16 sequences through the same layer: most experts are met
        _moe("moe_batch", tokens=16, H=4096, I=1536, experts=64, top=4, act="silu", renorm=True, kind="f32"),
        # an odd, larger batch through few wide experts, K ends inside a tile, probabilities over all experts
        _moe("moe_wide", tokens=61, H=3200, I=4320, experts=16, top=2, act="gelu", renorm=False, kind="f16"),
    ]


def draw(rng):
    def spread(low, high):
        return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))

    op = rng.choice(["quant", "gemm", "gemm", "gemm", "moe", "moe"])
    if op == "quant":
        K = 32 * spread(1, 344)
        return _quant(None, rows=spread(1, min(11008, int(MOST_CODED / 9.1 / K))), K=K, kind=rng.choice(["f16", "f32"]))
    if op == "gemm":
        N, K = spread(16, 11008), 32 * spread(2, 344)
        M = spread(1, 64) if rng.random() < 0.6 else spread(65, max(65, int(min(4096, MOST_FLOPS / 2 / N / K))))
        return _gemm(None, acts=rng.choice(["a16", "a8", "a4"]), M=M, N=N, K=K, out=rng.choice(["f16", "f16", "f32"]),
                     bias=rng.random() < 0.3)
    experts = spread(2, 128)
    H = 32 * spread(8, 128)
    I = 32 * spread(4, max(4, int(min(256, MOST_WEIGHTS / 0.54 / 3 / 32 / experts / H))))
    return _moe(None, tokens=1 if rng.random() < 0.3 else spread(2, 64), H=H, I=I, experts=experts,
                top=rng.randint(1, min(8, experts)), act=rng.choice(["silu", "silu", "gelu", "relu2"]),
                renorm=rng.random() < 0.6, kind=rng.choice(["f32", "f16"]))


def _case(op, name, c):
    return {"op": op, **({"name": name} if name else {}), **c}


def _quant(name, **c):
    return _case("quant", name, c)


def _gemm(name, **c):
    return _case("gemm", name, c)


def _moe(name, **c):
    return _case("moe", name, c)


def work(case):
    if case["op"] == "quant":
        n, b = case["rows"] * case["K"], 2 if case["kind"] == "f16" else 4
        return {"bytes": n * 2 * b + n / 2 + n / 32, "flops": 4 * n}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        rows = M * K * (1 if case["acts"] == "a8" else 2) + (4 * M if case["acts"] == "a8" else 0)
        return {"bytes": rows + N * K * (1 / 2 + 1 / 32) + M * N * (2 if case["out"] == "f16" else 4) + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, H, I, E, k = (case[x] for x in ("tokens", "H", "I", "experts", "top"))
    met = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, in the mean
    return {"bytes": met * 3 * H * I * (1 / 2 + 1 / 32) + T * E * (4 if case["kind"] == "f32" else 2) + 4 * T * H,
            "flops": 6 * T * k * H * I}


# ------------------------------------------------------------------ inputs
def _bits(e):
    """2.0 ** e for whole numbers -126 <= e <= 127."""
    return ((e + 127) << 23).view(torch.float32)


def _mx4(x):
    """Codes (uint8 [..., K / 2]) and scale bytes (uint8 [..., K / 32]) of float32 values."""
    blocks = x.unflatten(-1, (-1, 32))
    most = blocks.abs().amax(-1)
    e = torch.where(most > 0, (torch.frexp(most).exponent - 3).clamp(min=-126), -127)
    y = blocks * _bits(-e.clamp(min=-126))[..., None]
    a = y.abs()
    code = torch.signbit(y).to(torch.uint8) * 8
    # half way between two values: to the even code
    for middle, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += a >= middle if up else a > middle
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def weight(*shape):
        """Rows of an output channel each, some of them larger than others."""
        return _mx4(normal(*shape) * shape[-1] ** -0.5 * torch.exp(0.3 * normal(*shape[:-1], 1)))

    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    one = torch.cat([one, -one])
    state = {"case": case, "values": torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)}  # of a byte's two codes
    if case["op"] == "quant":
        gain = torch.exp(0.6 * normal(case["K"]))
        state["x"] = (normal(case["rows"], case["K"]) * gain).to(torch.float16 if case["kind"] == "f16" else torch.float32)
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        x = normal(M, K) * torch.exp(0.6 * normal(K))  # some channels of a residual stream are far larger than others
        if case["acts"] == "a8":
            scale = x.abs().amax(1) / 448
            state.update(codes=(x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale=scale)
        else:
            state["x"] = x.half()
        state["w"] = weight(N, K)
        state["bias"] = normal(N).half() if case["bias"] else None
        if own:
            import gemv_nibble_unpack_amd as G
            state.update(packed=G.prepack_mx4(*state["w"]), workspace=G.Workspace())
    else:
        T, H, I, E = (case[x] for x in ("tokens", "H", "I", "experts"))
        state["x"] = (normal(T, H) * torch.exp(0.3 * normal(H))).half()
        state["logits"] = (1.5 * normal(T, E)).to(torch.float16 if case["kind"] == "f16" else torch.float32)
        for name, n, k in (("w1", 2 * I, H), ("w2", H, I)):  # gate rows, then up rows; an expert at a time, for the memory
            each = [weight(n, k) for _ in range(E)]
            state[name] = tuple(torch.stack(x) for x in zip(*each))
        if own:
            import gemv_nibble_unpack_amd as G
            state.update(packed1=G.prepack_mx4(*(x.flatten(0, 1) for x in state["w1"])),
                         packed2=G.prepack_mx4(*(x.flatten(0, 1) for x in state["w2"])), workspace=G.Workspace())
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import gemv_nibble_unpack_amd as G
        return {"quant": _own_quant, "gemm": _own_gemm, "moe": _own_moe}[op](G, state)
    return {"quant": _plain_quant, "gemm": _plain_gemm, "moe": _plain_moe}[op](state)


def _own_quant(G, s):
    codes, scales = G.quantize_mx4(s["x"])
    return {"values": G.dequantize_mx4(codes, scales, s["x"].dtype), "scales": scales}


def _own_gemm(G, s):
    c = s["case"]
    more = {"bias": s["bias"], "out_dtype": G.W4_OUT_F16 if c["out"] == "f16" else G.W4_OUT_F32, "workspace": s["workspace"]}
    if c["acts"] == "a16":
        return G.mx4a16_gemm(s["x"], s["packed"], c["N"], **more)
    if c["acts"] == "a8":
        return G.mx4a8_gemm(s["codes"], s["scale"], s["packed"], c["N"], **more)
    codes, scales = G.quantize_mx4(s["x"])
    return G.mx4a4_gemm(codes, scales, s["packed"], c["N"], **more)


def _own_moe(G, s):
    c = s["case"]
    act = {"silu": G.W4_ACT_SILU, "gelu": G.W4_ACT_GELU, "relu2": G.W4_ACT_RELU2}[c["act"]]
    return G.moe_mx4(s["x"], s["logits"], c["top"], s["packed1"], s["packed2"], c["I"], act=act, renormalize=c["renorm"],
                     workspace=s["workspace"])


# ------------------------------------------------------------------ plain forms
def _values(s, codes, scales):
    """The float32 values of codes [..., K / 2] and scale bytes [..., K / 32] (no byte is 0 or 255 but in blocks of zeros)."""
    v = torch.index_select(s["values"], 0, codes.reshape(-1).int()).view(*scales.shape, 32)
    return (v * (scales.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def _plain_quant(s):
    codes, scales = _mx4(s["x"].float())
    return {"values": _values(s, codes, scales).to(s["x"].dtype), "scales": scales}


def _plain_gemm(s):
    c = s["case"]
    if c["acts"] == "a8":
        a = s["codes"].view(torch.float8_e4m3fn).float() * s["scale"][:, None]
    elif c["acts"] == "a16":
        a = s["x"].float()
    else:
        a = _values(s, *_mx4(s["x"].float()))
    y = torch.matmul(a, _values(s, *s["w"]).T)
    if s["bias"] is not None and c["out"] == "f16":  # float32 sums are handed on without it
        y = y + s["bias"].float()
    return y.to(torch.float16 if c["out"] == "f16" else torch.float32)


def _activation(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return torch.clamp(g, min=0) ** 2


def _plain_moe(s):
    c = s["case"]
    T, I, E, k = c["tokens"], c["I"], c["experts"], c["top"]
    logits, x = s["logits"].float(), s["x"].float()
    chosen = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    part = p.gather(1, chosen)
    part = part / (part if c["renorm"] else p).sum(1, keepdim=True)
    if T * k < E:  # the chosen experts' weights, one set for each choice
        at = chosen.flatten()
        w1, w2 = (_values(s, *(y[at] for y in s[n])) for n in ("w1", "w2"))
        h = torch.matmul(w1, x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        h = _activation(h[:, :I], c["act"]) * h[:, I:]
        y = torch.matmul(w2, h[:, :, None])[..., 0].view(T, k, -1)
        return (y * part[:, :, None]).sum(1).half()
    w1, w2 = (_values(s, *s[n]) for n in ("w1", "w2"))
    h = torch.matmul(x[None], w1.transpose(1, 2))  # every expert on every token
    h = _activation(h[..., :I], c["act"]) * h[..., I:]
    y = torch.matmul(h, w2.transpose(1, 2))
    share = torch.zeros(T, E, device="cuda").scatter_(1, chosen, part)
    return (y * share.T[:, :, None]).sum(0).half()


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_quant, "gemm": _exact_gemm, "moe": _exact_moe}[case["op"]](s)


def _decoded(codes, scales):
    """E2M1: sign, two bits of exponent (bias 1), one of mantissa; exponent 0 is subnormal."""
    def one(c):
        c = c.int()
        power, half = c >> 1 & 3, (c & 1).double() / 2
        size = torch.where(power == 0, half, (1 + half) * torch.exp2(power.double() - 1))
        return torch.where(c & 8 != 0, -size, size)

    v = torch.stack([one(codes & 15), one(codes >> 4)], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _nearest(x):
    """(values, scale bytes): each block's values as the nearest multiples of a step that grows with the magnitude, ties to the even one."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    most = b.abs().max(-1).values
    e = torch.where(most > 0, torch.floor(torch.log2(most.clamp(min=2.0 ** -140))) - 2, -127.0).clamp(min=-127)
    y = b / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)
    y = (torch.round(y / step) * step).clamp(-6, 6)
    return (y * torch.exp2(e)[..., None]).reshape(x.shape), (e + 127).to(torch.uint8)


def _exact_quant(s):
    values, scales = _nearest(s["x"])
    return {"values": values, "scales": scales}


def _exact_gemm(s):
    c = s["case"]
    if c["acts"] == "a8":
        a = s["codes"].view(torch.float8_e4m3fn).double() * s["scale"].double()[:, None]
    else:
        a = s["x"].double() if c["acts"] == "a16" else _nearest(s["x"])[0]
    y = a @ _decoded(*s["w"]).T
    return y + s["bias"].double() if s["bias"] is not None and c["out"] == "f16" else y


def _exact_moe(s):
    c = s["case"]
    x, logits = s["x"].double(), s["logits"].double()
    p = torch.softmax(logits, 1)
    # an expert's rank among a token's: how many are larger, or as large and before it
    before = torch.arange(c["experts"], device="cuda")
    ahead = (logits[:, None, :] > logits[:, :, None]) | ((logits[:, None, :] == logits[:, :, None]) & (before[None, :] < before[:, None])[None])
    p = torch.where(ahead.sum(2) < c["top"], p, 0.0)
    if c["renorm"]:
        p = p / p.sum(1, keepdim=True)
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        rows = torch.nonzero(p[:, e])[:, 0]
        if len(rows):
            g, u = (x[rows] @ _decoded(s["w1"][0][e], s["w1"][1][e]).T).split(c["I"], 1)
            if c["act"] == "silu":
                g = g * torch.sigmoid(g)
            elif c["act"] == "gelu":
                g = torch.nn.functional.gelu(g, approximate="tanh")
            else:
                g = torch.relu(g).square()
            out[rows] += p[rows, e, None] * ((g * u) @ _decoded(s["w2"][0][e], s["w2"][1][e]).T)
    return out
