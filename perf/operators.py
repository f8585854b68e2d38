"""What the block-scaled 8-bit operators are measured on.

Three operators that a serving program runs one after the other:

* ``quantize``: 16-bit activations or weights to 8-bit floating point with one
  fp32 scale for each block of 128 columns (1 x 128 for activations, 128 x 128
  for weights): scale = largest magnitude of the block / largest finite 8-bit
  value, code = value / scale rounded to nearest even.
* ``gemm``: y = A W^T of two such matrices, A [M][K] with 1 x 128 blocks and
  W [N][K] with 128 x 128 blocks.
* ``moe``: a whole mixture-of-experts layer for a few tokens: router logits,
  softmax, the top_k experts, each expert's silu(gate) * up and down products
  from 128 x 128-block 8-bit weights, and the weighted sum.

``run`` is the plain form (elementary torch operations in fp32, one rounding at
the end) while ``own`` is false and the package's calls while it is true.
``exact`` gives the operators' definition in fp64.
"""
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token's activations before a projection: latency only
        dict(name="quantize-token", op="quantize", rows=1, cols=4096, block_rows=1, x="fp16", code="e4m3"),
        # a prompt's activations before a 13B model's down projection
        dict(name="quantize-prompt", op="quantize", rows=4096, cols=13824, block_rows=1, x="bf16", code="e4m3"),
        # a weight matrix with odd edges in both directions, as a loader quantizes it
        dict(name="quantize-weight", op="quantize", rows=11000, cols=4100, block_rows=128, x="fp16", code="e4m3"),
        # one token through a 7B model's square projection: weight streaming, latency
        dict(name="gemm-token", op="gemm", m=1, n=4096, k=4096, y="fp16", a="e4m3", w="e4m3"),
        # a decode batch through a 13B model's down projection
        dict(name="gemm-batch16", op="gemm", m=16, n=5120, k=13824, y="bf16", a="e4m3", w="e4m3"),
        # a short ragged prompt, K not a whole number of blocks
        dict(name="gemm-ragged", op="gemm", m=333, n=5000, k=4104, y="bf16", a="e4m3", w="e4m3"),
        # a long prompt through a 7B model's up projection
        dict(name="gemm-prompt", op="gemm", m=8192, n=11008, k=4096, y="bf16", a="e4m3", w="e4m3"),
        # codes of the wide-range type, fp32 result
        dict(name="gemm-e5m2-fp32", op="gemm", m=1024, n=4096, k=4096, y="fp32", a="e5m2", w="e4m3"),
        # one token, many small experts
        dict(name="moe-token-small", op="moe", tokens=1, experts=64, top_k=6, hidden=2048, inter=1408, x="bf16", renormalize=False),
        # one token, few large experts (7B-sized MLPs)
        dict(name="moe-token-large", op="moe", tokens=1, experts=8, top_k=2, hidden=4096, inter=11008, x="fp16", renormalize=True),
        # a decode batch over many experts: most weights of the layer are read
        dict(name="moe-batch8", op="moe", tokens=8, experts=128, top_k=8, hidden=4096, inter=1408, x="bf16", renormalize=True),
        # the largest batch, experts shared by several tokens, ragged inner size
        dict(name="moe-batch32-ragged", op="moe", tokens=32, experts=32, top_k=4, hidden=2560, inter=1008, x="fp16", renormalize=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "moe", "moe"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 8192), _log(rng, 100, 13824)
        return dict(op=op, rows=min(rows, max(1, 4096 * 13824 // cols)), cols=cols, block_rows=rng.choice([1, 1, 128]),
                    x=rng.choice(["fp16", "bf16"]), code=rng.choice(["e4m3", "e4m3", "e5m2"]))
    if op == "gemm":
        n, k = _log(rng, 200, 14000), _log(rng, 200, 14000)
        m = min(_log(rng, 1, 8192), max(1, 8192 * 11008 * 4096 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, y=rng.choice(["fp16", "bf16", "bf16", "fp32"]),
                    a=rng.choice(["e4m3", "e4m3", "e5m2"]), w=rng.choice(["e4m3", "e4m3", "e5m2"]))
    experts = _log(rng, 4, 128)
    hidden, inter = 16 * _log(rng, 32, 256), 16 * _log(rng, 16, 160)
    return dict(op=op, tokens=_log(rng, 1, 32), experts=experts, top_k=rng.randint(1, min(8, experts)), hidden=hidden,
                inter=inter, x=rng.choice(["fp16", "bf16"]), renormalize=rng.random() < 0.5)


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": 3 * r * c + 4 * _up(r, case["block_rows"]) * _up(c, 128), "flops": 3 * r * c}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["y"] == "fp32" else 2
        return {"bytes": m * k + n * k + 4 * _up(k, 128) * (m + _up(n, 128)) + out * m * n, "flops": 2 * m * n * k}
    t, e, h, i, top = (case[v] for v in ("tokens", "experts", "hidden", "inter", "top_k"))
    seen = e * (1 - (1 - top / e) ** t)  # experts that t tokens are expected to reach
    return {"bytes": int(seen * 3 * h * i * (1 + 4 / 16384)) + 2 * e * h + 4 * t * h,
            "flops": 2 * t * e * h + 6 * t * top * h * i}


# ------------------------------------------------------------------ inputs
def _codes(gen, shape, code, spread):
    """Random codes with the spread that quantized normal values have; rows on a 16-byte pitch."""
    pitch = _up(shape[-1], 16) * 16
    q = torch.empty((*shape[:-1], pitch), dtype=_CODES[code], device="cuda")
    flat = q.view(-1, pitch)
    step = max(1, (1 << 26) // pitch)
    for r in range(0, flat.shape[0], step):
        part = flat[r:r + step]
        v = torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.float16)
        part.copy_((v * spread).clamp_(-4 * spread, 4 * spread).to(_CODES[code]))
    return q[..., : shape[-1]]


def _scales(gen, shape, about):
    return about * (0.5 + torch.rand(shape, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        x = torch.randn((r, c), generator=gen, device="cuda")
        # activations have a few columns of far larger values
        x *= 1 + 30 * (torch.rand((1, c), generator=gen, device="cuda") < 0.005)
        s["x_in"] = x.to(_TYPES[case["x"]])
        s["q"] = torch.empty((r, _up(c, 16) * 16), dtype=_CODES[case["code"]], device="cuda")[:, :c]
        s["scale"] = torch.empty((_up(r, case["block_rows"]), _up(c, 128)), device="cuda")
        return s
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        spread = {"e4m3": 112.0, "e5m2": 14336.0}
        s["a_q"] = _codes(gen, (m, k), case["a"], spread[case["a"]])
        s["w_q"] = _codes(gen, (n, k), case["w"], spread[case["w"]])
        s["a_s"] = _scales(gen, (m, _up(k, 128)), 1 / spread[case["a"]])
        s["w_s"] = _scales(gen, (_up(n, 128), _up(k, 128)), k ** -0.5 / spread[case["w"]])
        s["out"] = torch.empty((m, n), dtype=_TYPES[case["y"]], device="cuda")
        return s
    t, e, h, i = (case[v] for v in ("tokens", "experts", "hidden", "inter"))
    dt = _TYPES[case["x"]]
    s["x_in"] = torch.randn((t, h), generator=gen, device="cuda").to(dt)
    s["router"] = (torch.randn((e, h), generator=gen, device="cuda") * (1.5 * h ** -0.5)).to(dt)
    s["w13"] = _codes(gen, (e, 2 * i, h), "e4m3", 112.0)
    s["w2"] = _codes(gen, (e, h, i), "e4m3", 112.0)
    s["s13"] = _scales(gen, (e, 2, _up(i, 128), _up(h, 128)), h ** -0.5 / 112)
    s["s2"] = _scales(gen, (e, _up(h, 128), _up(i, 128)), i ** -0.5 / 112)
    s["out"] = torch.empty((t, h), dtype=dt, device="cuda")
    s["ids"] = torch.empty((t, case["top_k"]), dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty((t, case["top_k"]), device="cuda")
    if own:
        from lut_dequant_gemv_b200 import binding as B
        s["moe"] = B.sqz_create_moe(s["router"], s["w13"], s["s13"], s["w2"], s["s2"], top_k=case["top_k"],
                                    renormalize=case["renormalize"])
        s["workspace"] = B.sqz_moe_workspace(s["moe"], t)
    return s


# --------------------------------------------------------------- the passes
def run(state):
    if own:
        from lut_dequant_gemv_b200 import binding as B
        if state["op"] == "quantize":
            B.sqz_fp8_quantize(state["x_in"], block_rows=state["block_rows"], q=state["q"], scale=state["scale"])
            return {"q": state["q"], "scale": state["scale"]}
        if state["op"] == "gemm":
            B.sqz_fp8_gemm(state["a_q"], state["a_s"], state["w_q"], state["w_s"], state["out"])
            return {"y": state["out"]}
        B.sqz_moe_forward(state["moe"], state["x_in"], state["out"], ids=state["ids"], weights=state["weights"],
                          workspace=state["workspace"])
        return {"y": state["out"], "ids": state["ids"], "weights": state["weights"]}
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "moe": _plain_moe}[state["op"]](state)


def _plain_quantize(s):
    x = s["x_in"].float()
    (r, c), br = x.shape, s["block_rows"]
    x = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % br))
    x = x.view(x.shape[0] // br, br, x.shape[1] // 128, 128)
    scale = x.abs().amax(dim=(1, 3)) / _LARGEST[s["code"]]
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (x / scale[:, None, :, None]).reshape(x.shape[0] * br, -1)[:r, :c].to(_CODES[s["code"]])
    return {"q": q, "scale": scale}


def _spread_blocks(scale, rows, cols, block_rows):
    """One scale per element of the last two axes."""
    if block_rows > 1:
        scale = scale.repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return scale.repeat_interleave(128, dim=-1)[..., :cols]


def _plain_gemm(s):
    m, n, k = s["m"], s["n"], s["k"]
    a = s["a_q"].float() * _spread_blocks(s["a_s"], m, k, 1)
    w = s["w_q"].float() * _spread_blocks(s["w_s"], n, k, 128)
    return {"y": (a @ w.t()).to(s["out"].dtype)}


def _plain_moe(s):
    t, e, h, i, top = s["tokens"], s["experts"], s["hidden"], s["inter"], s["top_k"]
    x = s["x_in"].float()
    logits = x.double() @ s["router"].double().t()  # in 64 bits: the choice of experts is a border
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top]
    weights = torch.softmax(logits, dim=1).gather(1, order)
    if s["renormalize"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    weights = weights.float()
    if t * top < e:  # the experts of each pair
        at, xs = order.reshape(-1), x.repeat_interleave(top, dim=0)[:, :, None]
        w13, s13, w2, s2 = s["w13"][at], s["s13"][at], s["w2"][at], s["s2"][at]
    else:  # every expert, for all tokens
        xs, w13, s13, w2, s2 = x.t().expand(e, h, t), s["w13"], s["s13"], s["w2"], s["s2"]
    p = w13.shape[0]
    w13 = w13.float().view(p, 2, i, h) * _spread_blocks(s13, i, h, 128)
    both = torch.bmm(w13.view(p, 2 * i, h), xs)
    gate, up = both[:, :i], both[:, i:]
    hid = gate * torch.sigmoid(gate) * up
    out = torch.bmm(w2.float() * _spread_blocks(s2, h, i, 128), hid)  # [p, h, columns]
    if t * top < e:
        y = (out.view(t, top, h) * weights[:, :, None]).sum(dim=1)
    else:
        mix = torch.zeros((t, e), device=x.device).scatter_(1, order, weights)
        y = torch.einsum("eht,te->th", out, mix)
    return {"y": y.to(s["out"].dtype), "ids": order.to(torch.int32), "weights": weights}


# ------------------------------------------------------ the definition, fp64
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"quantize": _exact_quantize, "gemm": _exact_gemm, "moe": _exact_moe}[case["op"]](s)


def _exact_quantize(s):
    x, br, code = s["x_in"].double(), s["block_rows"], s["code"]
    r, c = x.shape
    scale = torch.ones((_up(r, br), _up(c, 128)), dtype=torch.float64, device=x.device)
    q = torch.zeros_like(x)
    mantissa, lowest = (3, -6) if code == "e4m3" else (2, -14)
    for j in range(_up(c, 128)):
        cols = x[:, 128 * j: 128 * j + 128]
        big = torch.nn.functional.pad(cols.abs().amax(dim=1), (0, -r % br)).view(-1, br).amax(dim=1)
        scale[:, j] = torch.where(big > 0, big / _LARGEST[code], scale[:, j])
        v = cols / scale[:, j].repeat_interleave(br)[:r, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** lowest))) - mantissa)
        q[:, 128 * j: 128 * j + 128] = torch.round(v / step) * step
    return {"q": q, "scale": scale}


def _exact_gemm(s):
    y = torch.zeros((s["m"], s["n"]), dtype=torch.float64, device="cuda")
    rows = torch.arange(s["n"], device="cuda") // 128
    for j in range(_up(s["k"], 128)):
        part = s["a_q"][:, 128 * j: 128 * j + 128].double() @ s["w_q"][:, 128 * j: 128 * j + 128].double().t()
        y += part * s["a_s"][:, j, None].double() * s["w_s"][rows, j].double()
    return {"y": y}


def _exact_moe(s):
    t, h, i, top = s["tokens"], s["hidden"], s["inter"], s["top_k"]
    x = s["x_in"].double()
    logits = x @ s["router"].double().t()
    prob = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    prob = prob / prob.sum(dim=1, keepdim=True)
    ids = torch.empty((t, top), dtype=torch.int64)
    weights = torch.zeros((t, top), dtype=torch.float64, device=x.device)
    left = logits.clone()
    for j in range(top):
        best = left.amax(dim=1, keepdim=True)
        at = (left == best).to(torch.int8).argmax(dim=1)  # the lowest index of a tie
        ids[:, j] = at.cpu()
        weights[:, j] = prob[torch.arange(t), at]
        left[torch.arange(t), at] = -torch.inf
    if s["renormalize"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    row_h, row_i = torch.arange(h, device=x.device) // 128, torch.arange(i, device=x.device) // 128
    y = torch.zeros((t, h), dtype=torch.float64, device=x.device)
    for e in sorted(set(ids.reshape(-1).tolist())):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        tok, slot = tok.to(x.device), slot.to(x.device)
        w1 = s["w13"][e, :i].double() * s["s13"][e, 0].double()[row_i][:, row_h]
        w3 = s["w13"][e, i:].double() * s["s13"][e, 1].double()[row_i][:, row_h]
        w2 = s["w2"][e].double() * s["s2"][e].double()[row_h][:, row_i]
        gate, up = x[tok] @ w1.t(), x[tok] @ w3.t()
        y.index_add_(0, tok, (gate / (1 + torch.exp(-gate)) * up) @ w2.t() * weights[tok, slot, None])
    return {"y": y, "ids": ids.to(torch.int32), "weights": weights}
