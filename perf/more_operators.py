"""Measured cases of the 4-bit operators beside the quantize: the MXFP4 cast and its reading back, the product of 4-bit
operands (NVFP4 and MXFP4), and a whole layer of gated experts for a few tokens over 4-bit weights.

Each case is one call (for the cast: the cast and the reading back of what it wrote) as a user's program makes it.
``run`` computes it in plain torch, in 32 bits, or, where ``own`` is set, through the package's entry points; ``exact``
computes the same outputs from the definitions in 64 bits.

Conventions (the package's own): E2M1 codes, two in a byte, the lower index in the low nibble, along the contracted
dimension.  "nvfp4": an E4M3 scale for each block of 16 and an amax (one per matrix or one per row), a value is
code * scale * (amax / 2688).  "mxfp4": a power-of-two scale for each block of 32, stored as its exponent + 127.  Scales
are compact, [rows, cols / block], or swizzled: tiles of 128 rows x 4 scales, 512 bytes each, where both dimensions are
multiples of 128.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # the tokens of one small decoding batch: latency is all that counts
        {"name": "cast_tokens", "op": "cast", "rows": 7, "cols": 4096, "dtype": "bf16", "colwise": False,
         "swizzled": False},
        # activations of a training batch, both directions, scales laid out for the product
        {"name": "cast_activations", "op": "cast", "rows": 8192, "cols": 5120, "dtype": "bf16", "colwise": True,
         "swizzled": True},
        # 32-bit master weights whose sizes fill no whole tile, compact scales
        {"name": "cast_weights", "op": "cast", "rows": 2080, "cols": 4128, "dtype": "fp32", "colwise": True,
         "swizzled": False},
        # one token through one weight matrix: bound by reading the weights
        {"name": "product_token", "op": "product", "format": "nvfp4", "m": 1, "n": 5120, "k": 4096, "per_row": False,
         "a_swizzled": False, "b_swizzled": True, "out": "bf16"},
        # odd sizes, a last block that half fills a step, compact scales, 32-bit output
        {"name": "product_ragged", "op": "product", "format": "mxfp4", "m": 333, "n": 1091, "k": 2080,
         "per_row": False, "a_swizzled": False, "b_swizzled": False, "out": "fp32"},
        # a prefill of some hundred tokens, each with its own amax
        {"name": "product_prefill", "op": "product", "format": "nvfp4", "m": 500, "n": 4096, "k": 4096,
         "per_row": True, "a_swizzled": False, "b_swizzled": True, "out": "bf16"},
        # a training batch through one weight matrix
        {"name": "product_train", "op": "product", "format": "nvfp4", "m": 8192, "n": 5120, "k": 8192,
         "per_row": False, "a_swizzled": True, "b_swizzled": True, "out": "bf16"},
        # a weight gradient: contracted along the tokens, 32-bit output
        {"name": "product_wgrad", "op": "product", "format": "mxfp4", "m": 5120, "n": 4096, "k": 16384,
         "per_row": False, "a_swizzled": True, "b_swizzled": True, "out": "fp32"},
        # one token through its experts: bound by reading their weights
        {"name": "experts_token", "op": "experts", "format": "nvfp4", "tokens": 1, "topk": 2, "experts": 8,
         "hidden": 4096, "inner": 2048},
        # a decoding batch, power-of-two scales, sizes that fill no whole step
        {"name": "experts_decode", "op": "experts", "format": "mxfp4", "tokens": 13, "topk": 4, "experts": 16,
         "hidden": 2720, "inner": 1184},
        # the largest decoding batch: every expert has several rows
        {"name": "experts_batch", "op": "experts", "format": "nvfp4", "tokens": 64, "topk": 4, "experts": 32,
         "hidden": 4096, "inner": 1536},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 5e12, w["flops"] / 5e13)


def draw(rng):
    most = max(_cost(c) for c in listed()) * 0.99
    while True:
        op = rng.choice(["cast", "product", "product", "experts", "experts"])
        if op == "cast":
            colwise = rng.random() < 0.6
            rows, cols = _log(rng, 1, 8192), 32 * _log(rng, 2, 256)
            rows = 32 * max(1, rows // 32) if colwise else rows
            c = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "fp32"]), "colwise": colwise,
                 "swizzled": rows % 128 == 0 and cols % 128 == 0}
        elif op == "product":
            m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), 32 * _log(rng, 4, 512)
            if rng.random() < 0.5:  # layer sizes are more often whole tiles
                n, k = 128 * max(1, n // 128), 128 * max(1, k // 128)
            if rng.random() < 0.3:
                m = 128 * max(1, m // 128)
            f = rng.choice(["nvfp4", "mxfp4"])
            c = {"op": op, "format": f, "m": m, "n": n, "k": k, "per_row": f == "nvfp4" and rng.random() < 0.4,
                 "a_swizzled": m % 128 == 0 and k % 128 == 0, "b_swizzled": n % 128 == 0 and k % 128 == 0,
                 "out": rng.choice(["bf16", "fp32"])}
        else:
            experts = rng.randint(2, 32)
            c = {"op": op, "format": rng.choice(["nvfp4", "mxfp4"]), "tokens": _log(rng, 1, 64),
                 "topk": rng.randint(1, min(8, experts)), "experts": experts, "hidden": 32 * _log(rng, 8, 192),
                 "inner": 32 * _log(rng, 4, 128)}
            if experts * c["hidden"] * c["inner"] > 32 * 4096 * 1536:
                continue
        if _cost(c) <= most:
            return c


# ---------------------------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------------------------
def _operand_bytes(fmt, rows, cols):
    return rows * cols // 2 + rows * cols // (16 if fmt == "nvfp4" else 32)


def work(case):
    op = case["op"]
    if op == "cast":
        n, dirs = case["rows"] * case["cols"], 1 + case["colwise"]
        # the cast reads x and writes codes and scales; reading back reads those and writes BF16 values
        coded = dirs * _operand_bytes("mxfp4", case["rows"], case["cols"])
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 2 * coded + dirs * n * 2, "flops": 3 * dirs * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _operand_bytes(case["format"], m, k) + _operand_bytes(case["format"], n, k) +
                m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    t, j, e, h, f = case["tokens"], case["topk"], case["experts"], case["hidden"], case["inner"]
    used = e * (1 - (1 - j / e) ** t)  # experts that some token chooses, on average
    return {"bytes": int(used * 3 * _operand_bytes(case["format"], h, f)) + t * (4 * h + 8 * j),
            "flops": 2 * t * j * 3 * h * f}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _e2m1(v):
    """Codes of the nearest E2M1 values (ties to the even code, at most 6)."""
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    for limit, inclusive in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= limit) if inclusive else (a > limit)
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _power(e):
    """2^e of whole numbers -1022 .. 1023, in 64 bits and from the bits: powers by pow() may be off by a unit, which
    decides ties."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _pack(code):
    return code[..., ::2] | (code[..., 1::2] << 4)


def _unpack(data):
    """The values of packed codes, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=data.device)
    return table[torch.stack([data & 15, data >> 4], -1).flatten(-2).int()]


def _swizzle(scale):
    r, c = scale.shape
    return scale.view(r // 128, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(r, c)


def _unswizzle(scale):
    r, c = scale.shape
    return scale.view(r // 128, c // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r, c)


def _mx_cast(x):
    """Codes [rows, cols] (one in a byte) and exponents + 127 [rows, cols / 32] of the MXFP4 cast of x: the largest
    power of two not above the block's maximum, over 4."""
    rows, cols = x.shape
    f = x.float().view(rows, cols // 32, 32)
    amax = f.abs().amax(-1)
    exponent = (torch.frexp(amax).exponent - 3 + 127).clamp(min=0, max=254)
    exponent = torch.where(amax == 0, torch.zeros_like(exponent), exponent)
    fine = torch.isfinite(amax)
    v = f * _power(127 - exponent).float()[..., None]
    code = torch.where(fine[..., None], _e2m1(v), torch.zeros((), dtype=torch.uint8, device=x.device))
    return code.view(rows, cols), torch.where(fine, exponent, 255).to(torch.uint8)


def _nv_cast(x, per_row):
    """The same of the NVFP4 cast, with its amax."""
    rows, cols = x.shape
    f = x.float()
    amax = f.abs().amax(1) if per_row else f.abs().max().view(1)
    g = torch.where(amax == 0, 1.0, 2688.0 / amax)[:, None]
    f = f.view(rows, cols // 16, 16)
    scale = (f.abs().amax(-1) / 6.0 * g).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    code = _e2m1(f * torch.where(s == 0, 0.0, g / s)[..., None])
    return code.view(rows, cols), scale.view(torch.uint8), amax


def _operand(x, fmt, per_row=False, swizzled=False):
    """Packed codes, scales and amax (or None) of x, made as a user's earlier cast made them."""
    code, scale, amax = _nv_cast(x, per_row) if fmt == "nvfp4" else _mx_cast(x) + (None,)
    return _pack(code), _swizzle(scale) if swizzled else scale, amax


def _experts(shape, std, fmt, g):
    """The operands of a stack of weight matrices, each with its own amax."""
    each = [_operand(_normal(shape[1:], g, std), fmt) for _ in range(shape[0])]
    amax = torch.cat([a for _, _, a in each]) if fmt == "nvfp4" else None
    return torch.stack([d for d, _, _ in each]), torch.stack([s for _, s, _ in each]), amax


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op == "cast":
        x = _normal((case["rows"], case["cols"]), g)
        hot = torch.rand(x.shape, generator=g, device="cuda") < 1e-3  # a few large values, as activations have
        s["x"] = torch.where(hot, x * 30.0, x).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        return s
    fmt = case["format"]
    if op == "product":
        s["a"] = _operand(_normal((case["m"], case["k"]), g), fmt, case["per_row"], case["a_swizzled"])
        s["b"] = _operand(_normal((case["n"], case["k"]), g, 0.02), fmt, False, case["b_swizzled"])
        return s
    t, j, e, h, f = case["tokens"], case["topk"], case["experts"], case["hidden"], case["inner"]
    # gate rows, then up rows, of each expert; and the matrix back to the hidden size
    s["gate_up"] = _experts((e, 2 * f, h), h ** -0.5, fmt, g)
    s["down"] = _experts((e, h, f), f ** -0.5, fmt, g)
    s["x"] = _normal((t, h), g, 1.0, torch.bfloat16)
    # a token's choices: distinct, some experts better liked than others, about 1 in 100 dropped by a capacity limit
    logits = _normal((t, e), g) + _normal((1, e), g, 0.3)
    top = torch.topk(logits, j, 1)
    drop = torch.rand((t, j), generator=g, device="cuda") < 0.01
    s["ids"] = torch.where(drop, -1, top.indices).to(torch.int32)
    s["gates"] = torch.softmax(top.values, 1)
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _values(operand, swizzled=False):
    """What a matrix of codes stands for, in 32 bits."""
    data, scale, amax = operand
    v = _unpack(data)
    rows, cols = v.shape
    if swizzled:
        scale = _unswizzle(scale)
    if amax is None:
        s = _power(scale.int() - 127).float()
        s = torch.where(scale == 255, math.nan, s)
    else:
        s = scale.view(torch.float8_e4m3fn).float()
    v = (v.view(rows, s.shape[1], -1) * s[..., None]).view(rows, cols)
    return v if amax is None else v * (amax / 2688.0)[:, None]


def _plain(s):
    op = s["op"]
    if op == "cast":
        out = {}
        for name in ("row", "col") if s["colwise"] else ("row",):
            x = s["x"] if name == "row" else s["x"].t().contiguous()
            code, scale = _mx_cast(x)
            out[name] = _values((_pack(code), scale, None)).to(torch.bfloat16)
            out[name + "_scale"] = _swizzle(scale) if s["swizzled"] else scale
        return out
    if op == "product":
        dtype = torch.bfloat16 if s["out"] == "bf16" else torch.float32
        return (_values(s["a"], s["a_swizzled"]) @ _values(s["b"], s["b_swizzled"]).t()).to(dtype)
    # every token through every expert, weighted by the gates of its choices (0 where there is none)
    e, f = s["experts"], s["inner"]
    part = lambda op, i: tuple(None if v is None else v[i:i + 1] if v.dim() == 1 else v[i] for v in op)  # noqa: E731
    x, ids = s["x"].float(), s["ids"].long()
    y = torch.zeros_like(x)
    for i in range(e):
        w = torch.where(ids == i, s["gates"], 0.0).sum(1)
        chosen = (ids == i).any(1)
        u = x @ _values(part(s["gate_up"], i)).t()
        h = u[:, :f] * torch.sigmoid(u[:, :f]) * u[:, f:]
        z = h @ _values(part(s["down"], i)).t()
        y += torch.where(chosen[:, None], z * w[:, None], 0.0)
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import nvfp4_block_scaled_amax_gb300 as nv
    op = s["op"]
    if op == "cast":
        q = nv.quantize_mxfp4(s["x"], colwise=s["colwise"], swizzled=s["swizzled"])
        out = {"row": nv.dequantize_fp4(q.row), "row_scale": q.row.scale.view(s["rows"], -1)}
        if s["colwise"]:
            out["col"], out["col_scale"] = nv.dequantize_fp4(q.col), q.col.scale.view(s["cols"], -1)
        return out
    block = 16 if s["format"] == "nvfp4" else 32
    if op == "product":
        a = nv.FP4Operand(*s["a"], block=block, swizzled=s["a_swizzled"])
        b = nv.FP4Operand(*s["b"], block=block, swizzled=s["b_swizzled"])
        return nv.matmul_fp4(a, b, out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    return nv.expert_mlp(s["x"], nv.FP4Operand(*s["gate_up"], block=block), nv.FP4Operand(*s["down"], block=block),
                         s["ids"], s["gates"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_values(operand, block, swizzled):
    data, scale, amax = operand
    rows, cols = data.shape[0], 2 * data.shape[1]
    v = torch.empty((rows, cols), dtype=torch.float64, device=data.device)
    for half in range(2):
        code = (data.int() >> (4 * half)) & 15
        m, e = (code & 1).double(), (code >> 1) & 3
        a = torch.where(e == 0, m / 2, (1 + m / 2) * _power(e - 1))
        v[:, half::2] = torch.where(code >= 8, -a, a)
    r = torch.arange(rows, device=data.device)[:, None]
    c = torch.arange(cols // block, device=data.device)[None]
    at = ((r // 128) * (cols // block // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4 if swizzled else \
        r * (cols // block) + c
    byte = scale.reshape(-1)[at].int()
    if amax is None:
        s = _power(byte - 127)
        s[byte == 255] = math.nan
    else:
        m, e = (byte & 7).double(), byte >> 3
        s = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * _power(e - 7))
        s = s * (amax.double() / 2688)[:, None]
    return v * s.repeat_interleave(block, 1)


def _exact_cast(x):
    """The MXFP4 value of each element of x along its rows."""
    rows, cols = x.shape
    v = x.double().reshape(rows, cols // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    shared = (amax.view(torch.int64) >> 52) - 1023  # the exponent field: log2() may round past a power of two
    unit = _power((shared - 2).clamp(min=-127))
    p = (v / unit).abs().clamp(max=6.0)
    step = torch.where(p < 2, 0.5, torch.where(p < 4, 1.0, 2.0))
    return (torch.copysign((p / step).round() * step, v) * unit).reshape(rows, cols)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "cast":
        out = {}
        for name in ("row", "col") if case["colwise"] else ("row",):
            out[name], out[name + "_scale"] = _exact_cast(s["x"] if name == "row" else s["x"].t()), None
        return out
    block = 16 if case["format"] == "nvfp4" else 32
    if op == "product":
        return _exact_values(s["a"], block, case["a_swizzled"]) @ _exact_values(s["b"], block, case["b_swizzled"]).t()
    t, f = case["tokens"], case["inner"]
    y = torch.zeros((t, case["hidden"]), dtype=torch.float64, device="cuda")
    ids = s["ids"].tolist()
    for i in sorted({e for row in ids for e in row if e >= 0}):
        up, down = ([v if v is None else v[i].reshape(1) if v.dim() == 1 else v[i] for v in s[name]]
                    for name in ("gate_up", "down"))
        w_up, w_down = _exact_values(up, block, False), _exact_values(down, block, False)
        at = [(r, j) for r, row in enumerate(ids) for j, e in enumerate(row) if e == i]
        rows = torch.tensor([r for r, _ in at], device="cuda")
        gates = s["gates"][rows, torch.tensor([j for _, j in at], device="cuda")].double()
        u = s["x"][rows].double() @ w_up.t()
        h = u[:, :f] / (1 + torch.exp(-u[:, :f])) * u[:, f:]
        y.index_add_(0, rows, (h @ w_down.t()) * gates[:, None])
    return y
