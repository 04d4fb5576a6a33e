"""Measured cases of the expert-layer operators: tokens sorted by expert and back, the 8-bit cast with a scale for
each block of 128, and the 8-bit matrix product (dense, by expert, and its weight gradient).

Each case is one call (or one training step's pair of calls) as a user's program makes it.  ``run`` computes it in
plain torch, in 32 bits, or, where ``own`` is set, through the package's entry points; ``exact`` computes the same
outputs from the definitions in 64 bits.

Conventions (the package's own): a scale covers 128 consecutive elements along the contracted dimension, for one row
("block_rows" 1, scales [ceil(K/128), rows]) or for 128 rows ("block_rows" 128, scales [ceil(rows/128), ceil(K/128)]).
"""
import math

import torch

own = False

BLOCK = 128
AMAX_FLOOR = 2.0 ** -100  # a block whose values are all smaller is scaled as if its maximum were this


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a small batch: latency is all that counts
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 8, "topk": 2, "experts": 8, "width": 1024, "align": 1},
        # a training batch sent to its experts, members padded to 128 rows for the cast along the tokens
        {"name": "dispatch_train", "op": "dispatch", "tokens": 16384, "topk": 4, "experts": 32, "width": 4096,
         "align": 128},
        # the experts' rows of an odd-sized serving batch joined back into tokens
        {"name": "combine_serve", "op": "combine", "tokens": 101, "topk": 2, "experts": 16, "width": 5120, "align": 1,
         "grad": False},
        # a training batch joined, and its gradients: rows and weights
        {"name": "combine_train", "op": "combine", "tokens": 8192, "topk": 4, "experts": 32, "width": 5120,
         "align": 128, "grad": True},
        # activations of a training batch, both directions (forward product and weight gradient)
        {"name": "cast_activations", "op": "cast", "batch": 1, "rows": 8192, "cols": 5120, "dtype": "bf16",
         "block_rows": 1, "colwise": True},
        # 32-bit master weights of several experts, 128 x 128 blocks, last row block half filled
        {"name": "cast_weights", "op": "cast", "batch": 4, "rows": 2112, "cols": 4096, "dtype": "fp32",
         "block_rows": 128, "colwise": True},
        # one token through one weight matrix: bound by reading the weights
        {"name": "product_token", "op": "product", "m": 1, "n": 5120, "k": 4096, "block_rows": 128, "out": "bf16"},
        # odd sizes, a short last block, a scale per weight row, 32-bit output
        {"name": "product_ragged", "op": "product", "m": 333, "n": 1091, "k": 2064, "block_rows": 1, "out": "fp32"},
        # a training batch through one weight matrix
        {"name": "product_train", "op": "product", "m": 8192, "n": 5120, "k": 8192, "block_rows": 128, "out": "bf16"},
        # a decoding batch through its experts: few rows each, bound by reading the touched weights
        {"name": "experts_decode", "op": "experts", "rows": 64, "experts": 16, "n": 4096, "k": 2048, "align": 1,
         "block_rows": 128, "out": "bf16"},
        # the same for a training batch: every expert's rows through its own weights
        {"name": "experts_train", "op": "experts", "rows": 16384, "experts": 16, "n": 2048, "k": 4096, "align": 128,
         "block_rows": 128, "out": "bf16"},
        # the experts' weight gradients of a training batch
        {"name": "experts_wgrad", "op": "wgrad", "rows": 16384, "experts": 8, "n": 4096, "k": 2048, "align": 128,
         "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 5e12, w["flops"] / 5e13)


def draw(rng):
    most = max(_cost(c) for c in listed()) * 0.99
    while True:
        op = rng.choice(["dispatch", "combine", "cast", "product", "experts", "wgrad"])
        if op in ("dispatch", "combine"):
            c = {"op": op, "tokens": _log(rng, 1, 16384), "topk": rng.randint(1, 8), "experts": rng.randint(2, 128),
                 "width": 8 * _log(rng, 8, 1024), "align": rng.choice([1, 16, 128])}
            if op == "combine":
                c["grad"] = rng.random() < 0.6
        elif op == "cast":
            colwise = rng.random() < 0.6
            rows = _log(rng, 1, 8192)
            c = {"op": op, "batch": rng.choice([1, 1, 2, 5]), "rows": 16 * max(1, rows // 16) if colwise else rows,
                 "cols": 16 * _log(rng, 4, 512), "dtype": rng.choice(["bf16", "fp32"]),
                 "block_rows": rng.choice([1, 128]), "colwise": colwise}
        elif op == "product":
            c = {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 8192), "k": 16 * _log(rng, 8, 512),
                 "block_rows": rng.choice([1, 128]), "out": rng.choice(["bf16", "fp32"])}
        elif op == "experts":
            c = {"op": op, "rows": _log(rng, 1, 16384), "experts": rng.randint(2, 32), "n": 8 * _log(rng, 16, 640),
                 "k": 16 * _log(rng, 16, 256), "align": rng.choice([1, 128]), "block_rows": rng.choice([1, 128]),
                 "out": rng.choice(["bf16", "fp32"])}
        else:
            c = {"op": op, "rows": _log(rng, 64, 16384), "experts": rng.randint(2, 8), "n": 8 * _log(rng, 16, 512),
                 "k": 8 * _log(rng, 16, 384), "align": 128, "out": rng.choice(["bf16", "fp32"])}
        if _cost(c) <= most:
            return c


# ---------------------------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------------------------
def _blocks(n):
    return -(-n // BLOCK)


def _capacity(slots, experts, align):
    return (slots + experts * (align - 1)) // align * align


def _scale_count(batch, rows, cols, block_rows):
    return batch * _blocks(cols) * (rows if block_rows == 1 else _blocks(rows))


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine"):
        t, k, h = case["tokens"], case["topk"], case["width"]
        r = _capacity(t * k, case["experts"], case["align"])
        if op == "dispatch":  # ids and tokens in; rows, both maps and the offsets out
            return {"bytes": t * k * 4 + t * h * 2 + r * h * 2 + t * k * 4 + r * 4 + (case["experts"] + 1) * 4,
                    "flops": 0}
        nbytes, flops = t * k * (h * 2 + 8) + t * h * 2, 2 * t * k * h  # rows, map, weights in; tokens out
        if case["grad"]:  # the tokens' gradient (and, if not kept on the chip, the rows) in; both gradients out
            nbytes += t * h * 2 + r * h * 2 + r * 4 + t * k * 4
            flops += 3 * t * k * h
        return {"bytes": nbytes, "flops": flops}
    if op == "cast":
        b, m, n = case["batch"], case["rows"], case["cols"]
        dirs = 1 + case["colwise"]
        nbytes = b * m * n * ((2 if case["dtype"] == "bf16" else 4) + dirs) + 4 * _scale_count(b, m, n, case["block_rows"])
        if case["colwise"]:
            nbytes += 4 * _scale_count(b, n, m, case["block_rows"])
        return {"bytes": nbytes, "flops": 2 * dirs * b * m * n}
    out = 2 if case["out"] == "bf16" else 4
    n, k = case["n"], case["k"]
    if op == "product":
        m = case["m"]
        return {"bytes": m * k + n * k + 4 * (_scale_count(1, m, k, 1) + _scale_count(1, n, k, case["block_rows"])) +
                m * n * out, "flops": 2 * m * n * k}
    e = case["experts"]
    r = _capacity(case["rows"], e, case["align"])
    if op == "experts":
        used = min(e - (e > 4), case["rows"])  # experts that have rows at all
        return {"bytes": r * k + used * n * k + 4 * (_scale_count(1, r, k, 1) +
                _scale_count(used, n, k, case["block_rows"])) + r * n * out, "flops": 2 * case["rows"] * n * k}
    return {"bytes": r * (n + k) + 4 * _blocks(r) * (n + k) + e * n * k * out, "flops": 2 * case["rows"] * n * k}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _popularity(experts, g):
    """How much a router likes each expert: uneven, and one of more than four is never chosen."""
    p = 0.4 + torch.rand(experts, generator=g, device="cuda")
    if experts > 4:
        p[experts // 2] = 0.0
    return p


def _expert_ids(tokens, topk, experts, g):
    """Top-k choices of a router over uneven experts: distinct for a token while there are enough experts; about 1 in
    100 is -1 (dropped by a capacity limit)."""
    p = _popularity(experts, g)
    usable = int((p > 0).sum())
    if topk <= usable:
        ids = torch.multinomial(p.expand(tokens, experts).contiguous(), topk, generator=g)
    else:
        ids = torch.multinomial(p, tokens * topk, replacement=True, generator=g).view(tokens, topk)
    drop = torch.rand(tokens, topk, generator=g, device="cuda") < 0.01
    return torch.where(drop, torch.full_like(ids, -1), ids).to(torch.int32)


def _member_offsets(rows, experts, align, g):
    """First row of each expert's member and the end, every member a multiple of align rows, as the sort gives."""
    ids = torch.multinomial(_popularity(experts, g), rows, replacement=True, generator=g)
    count = torch.zeros(experts, dtype=torch.int64, device="cuda").scatter_add_(0, ids, torch.ones_like(ids))
    padded = (count + align - 1) // align * align
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return torch.cat([zero, padded.cumsum(0)]).to(torch.int32), count


def _operand(x, block_rows):
    """8-bit codes and scales of x along its last dimension, made as a user's earlier cast made them."""
    return _cast_plain(x, block_rows)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op in ("dispatch", "combine"):
        t, k, e, h = case["tokens"], case["topk"], case["experts"], case["width"]
        s["ids"] = _expert_ids(t, k, e, g)
        if op == "dispatch":
            s["x"] = _normal((t, h), g, 1.0, torch.bfloat16)
            return s
        s["offsets"], s["row_of_slot"], s["slot_of_row"] = _sort_plain(s["ids"], e, case["align"])
        s["rows"] = _normal((s["slot_of_row"].numel(), h), g, 0.5, torch.bfloat16)
        s["weights"] = torch.softmax(_normal((t, k), g), 1)
        if case["grad"]:
            s["dy"] = _normal((t, h), g, 1e-3, torch.bfloat16)
        return s
    if op == "cast":
        shape = (case["rows"], case["cols"]) if case["batch"] == 1 else (case["batch"], case["rows"], case["cols"])
        x = _normal(shape, g, 0.02 if case["block_rows"] == 128 else 1.0)
        hot = torch.rand(shape, generator=g, device="cuda") < 1e-3  # a few large values, as activations have
        x = torch.where(hot, x * 30.0, x)
        s["x"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        return s
    n, k = case["n"], case["k"]
    if op == "product":
        s["a"], s["a_scale"] = _operand(_normal((case["m"], k), g), 1)
        s["b"], s["b_scale"] = _operand(_normal((n, k), g, 0.02), case["block_rows"])
        return s
    e, align = case["experts"], case["align"]
    s["offsets"], count = _member_offsets(case["rows"], e, align, g)
    r = _capacity(case["rows"], e, align)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # rows of the fullest member
    row = torch.arange(r, device="cuda")
    first = s["offsets"][:-1].long()
    member = torch.searchsorted(s["offsets"][1:].long(), row, right=True).clamp(max=e - 1)
    real = row < first[member] + count[member]  # the padding rows of a member are zero
    if op == "experts":
        s["a"], s["a_scale"] = _operand(_normal((r, k), g) * real[:, None], 1)
        s["b"], s["b_scale"] = _operand(_normal((e, n, k), g, 0.02), case["block_rows"])
        return s
    s["a"], s["a_scale"] = _operand((_normal((r, n), g, 1e-3) * real[:, None]).t().contiguous(), 1)
    s["b"], s["b_scale"] = _operand((_normal((r, k), g) * real[:, None]).t().contiguous(), 1)
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _sort_plain(ids, experts, align):
    flat = ids.reshape(-1).long()
    slots = flat.numel()
    rows = _capacity(slots, experts, align)
    at = torch.arange(slots, device=flat.device)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (count[:experts] + align - 1) // align * align
    offsets = torch.cat([torch.zeros_like(count[:1]), padded.cumsum(0)])
    begin = count.cumsum(0) - count
    key = key[order]
    row = torch.where(key < experts, offsets[key] + at - begin[key], torch.full_like(key, -1))
    row_of_slot = torch.empty_like(row)
    row_of_slot[order] = row
    slot_of_row = torch.full((rows + 1,), -1, dtype=torch.int64, device=flat.device)
    slot_of_row[torch.where(row >= 0, row, torch.full_like(row, rows))] = order
    return offsets.to(torch.int32), row_of_slot.view(ids.shape).to(torch.int32), slot_of_row[:rows].to(torch.int32)


def _cast_plain(x, block_rows):
    """E4M3 codes of x with a scale for each block of 128 along the last dimension."""
    f = x.float()
    rows, cols = f.shape[-2:]
    nb = _blocks(cols)
    f = torch.nn.functional.pad(f, (0, nb * BLOCK - cols))
    f = f.view(*f.shape[:-1], nb, BLOCK)
    amax = f.abs().amax(-1)  # [.., rows, nb]
    if block_rows > 1:
        mb = _blocks(rows)
        padded = torch.nn.functional.pad(amax, (0, 0, 0, mb * BLOCK - rows))
        amax = padded.view(*amax.shape[:-2], mb, BLOCK, nb).amax(-2)
    amax = amax.clamp(min=AMAX_FLOOR)
    top = torch.full((), 448.0, device=x.device)
    scale, factor = amax / top, top / amax
    if block_rows > 1:
        factor = factor.repeat_interleave(BLOCK, -2)[..., :rows, :]
    q = (f * factor[..., None]).flatten(-2)[..., :cols].clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q, scale if block_rows > 1 else scale.transpose(-1, -2).contiguous()


def _values(q, scale, block_rows):
    """What the codes stand for, in 32 bits."""
    rows, cols = q.shape[-2:]
    if block_rows > 1:
        scale = scale.repeat_interleave(BLOCK, -2)[..., :rows, :]
    else:
        scale = scale.transpose(-1, -2)
    return q.float() * scale.repeat_interleave(BLOCK, -1)[..., :cols]


def _member_rows(s):
    """Rows of each member side by side, [experts, most], and which of them exist."""
    first, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    idx = first[:, None] + torch.arange(s["most"], device=first.device)
    return idx, idx < end[:, None]


def _plain(s):
    op = s["op"]
    if op == "dispatch":
        offsets, row_of_slot, slot_of_row = _sort_plain(s["ids"], s["experts"], s["align"])
        token = slot_of_row.clamp(min=0) // s["topk"]
        rows = torch.where((slot_of_row >= 0)[:, None], s["x"][token], torch.zeros_like(s["x"][:1]))
        return {"rows": rows, "offsets": offsets, "row_of_slot": row_of_slot, "slot_of_row": slot_of_row}
    if op == "combine":
        at, slot = s["row_of_slot"].long(), s["slot_of_row"].long()
        rows = torch.where((at >= 0)[..., None], s["rows"][at.clamp(min=0)].float(), 0.0)
        out = {"y": (rows * s["weights"][..., None]).sum(1).to(torch.bfloat16)}
        if s["grad"]:
            dy = s["dy"].float()
            out["dweights"] = (rows * dy[:, None]).sum(-1)
            w = torch.where(slot >= 0, s["weights"].reshape(-1)[slot.clamp(min=0)], 0.0)
            out["drows"] = (dy[slot.clamp(min=0) // s["topk"]] * w[:, None]).to(torch.bfloat16)
        return out
    if op == "cast":
        out = {}
        out["row"], out["row_scale"] = _cast_plain(s["x"], s["block_rows"])
        if s["colwise"]:
            out["col"], out["col_scale"] = _cast_plain(s["x"].transpose(-1, -2), s["block_rows"])
        return out
    dtype = torch.bfloat16 if s["out"] == "bf16" else torch.float32
    a = _values(s["a"], s["a_scale"], 1)
    b = _values(s["b"], s["b_scale"], s.get("block_rows", 1))
    if op == "product":
        return (a @ b.t()).to(dtype)
    idx, there = _member_rows(s)
    if op == "experts":
        r = a.shape[0]
        members = torch.where(there[..., None], a[idx.clamp(max=r - 1)], 0.0)
        y = torch.zeros((r + 1, s["n"]), device=a.device)
        y[torch.where(there, idx, torch.full_like(idx, r))] = torch.bmm(members, b.transpose(1, 2))
        return y[:r].to(dtype)
    cols = idx.clamp(max=a.shape[1] - 1)
    am = torch.where(there[:, None], a[:, cols].transpose(0, 1), 0.0)  # [experts, n, most]
    bm = torch.where(there[:, None], b[:, cols].transpose(0, 1), 0.0)  # [experts, k, most]
    return torch.bmm(am, bm.transpose(1, 2)).to(dtype)


# ---------------------------------------------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import nvfp4_block_scaled_amax_gb300 as nv
    op = s["op"]
    if op == "dispatch":
        rows, plan = nv.dispatch_tokens(s["x"], s["ids"], s["experts"], align=s["align"])
        return {"rows": rows, "offsets": plan.offsets, "row_of_slot": plan.row_of_slot,
                "slot_of_row": plan.slot_of_row}
    if op == "combine":
        plan = nv.TokenPlan(s["offsets"], s["row_of_slot"], s["slot_of_row"])
        out = {"y": nv.combine_tokens(s["rows"], plan, s["weights"])}
        if s["grad"]:
            out["drows"], out["dweights"] = nv.combine_tokens_grad(s["dy"], s["rows"], plan, s["weights"])
        return out
    if op == "cast":
        q = nv.quantize_fp8(s["x"], block_rows=s["block_rows"], colwise=s["colwise"])
        out = {"row": q.row.data, "row_scale": q.row.scale}
        if s["colwise"]:
            out["col"], out["col_scale"] = q.col.data, q.col.scale
        return out
    dtype = torch.bfloat16 if s["out"] == "bf16" else torch.float32
    a = nv.FP8Operand(s["a"], s["a_scale"])
    b = nv.FP8Operand(s["b"], s["b_scale"], block_rows=s.get("block_rows", 1))
    if op == "product":
        return nv.matmul_fp8(a, b, out_dtype=dtype)
    if op == "experts":
        return nv.matmul_fp8_grouped(a, b, s["offsets"], out_dtype=dtype)
    return nv.matmul_fp8_grouped_wgrad(a, b, s["offsets"], out_dtype=dtype)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_places(ids, experts, align):
    """Row of each slot and slot of each row, by walking the slots in order."""
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(experts)]
    for slot, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(slot)
    slot_of_row = []
    for members in lists:
        slot_of_row += members + [-1] * (-len(members) % align)
    slot_of_row += [-1] * (_capacity(len(flat), experts, align) - len(slot_of_row))
    row_of_slot = [-1] * len(flat)
    for row, slot in enumerate(slot_of_row):
        if slot >= 0:
            row_of_slot[slot] = row
    return (torch.tensor(row_of_slot, dtype=torch.int64, device="cuda").view(ids.shape),
            torch.tensor(slot_of_row, dtype=torch.int64, device="cuda"))


def _exact_e4m3(v):
    """The nearest E4M3 value, ties to even, at most 448."""
    a = v.abs().clamp(max=448.0)
    e = torch.frexp(a).exponent.clamp(min=-5) - 4  # three bits after the leading one; 2^-9 steps below 2^-6
    step = torch.ldexp(torch.ones_like(a), e)
    return torch.copysign(torch.round(a / step) * step, v)


def _exact_cast(x, block_rows):
    rows, cols = x.shape
    q = torch.empty_like(x)
    scales = []
    for c in range(0, cols, BLOCK):
        part = x[:, c:c + BLOCK]
        if block_rows == 1:
            amax = part.abs().amax(1).clamp(min=AMAX_FLOOR)
            q[:, c:c + BLOCK] = _exact_e4m3(part * (448.0 / amax)[:, None])
            scales.append(amax / 448.0)
        else:
            column = []
            for r in range(0, rows, BLOCK):
                amax = part[r:r + BLOCK].abs().max().clamp(min=AMAX_FLOOR)
                q[r:r + BLOCK, c:c + BLOCK] = _exact_e4m3(part[r:r + BLOCK] * (448.0 / amax))
                column.append(amax / 448.0)
            scales.append(torch.stack(column))
    scale = torch.stack(scales)  # [column blocks, rows or row blocks]
    return q, scale if block_rows == 1 else scale.t().contiguous()


def _exact_values(q, scale, block_rows):
    v = q.double()
    for b in range(_blocks(v.shape[1])):
        c = slice(b * BLOCK, (b + 1) * BLOCK)
        if block_rows == 1:
            v[:, c] *= scale[b].double()[:, None]
        else:
            for r in range(scale.shape[0]):
                v[r * BLOCK:(r + 1) * BLOCK, c] *= scale[r, b].double()
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        _, slot = _exact_places(s["ids"], case["experts"], case["align"])
        rows = torch.zeros((slot.numel(), case["width"]), dtype=torch.float64, device="cuda")
        real = slot >= 0
        rows[real] = s["x"].double()[slot[real] // case["topk"]]
        return {"rows": rows, "offsets": None, "row_of_slot": None, "slot_of_row": None}
    if op == "combine":
        row, slot = _exact_places(s["ids"], case["experts"], case["align"])
        w = s["weights"].double()
        y = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        for j in range(case["topk"]):
            there = row[:, j] >= 0
            part = s["rows"][row[there, j]].double()
            y[there] += w[there, j, None] * part
            if case["grad"]:
                dw[there, j] = (part * s["dy"][there].double()).sum(1)
        out = {"y": y}
        if case["grad"]:
            drows = torch.zeros((slot.numel(), case["width"]), dtype=torch.float64, device="cuda")
            real = slot >= 0
            drows[real] = w.view(-1)[slot[real], None] * s["dy"].double()[slot[real] // case["topk"]]
            out["dweights"], out["drows"] = dw, drows
        return out
    if op == "cast":
        parts = s["x"].double().view(case["batch"], case["rows"], case["cols"])
        out = {}
        for name in ("row", "col") if case["colwise"] else ("row",):
            each = [_exact_cast(p if name == "row" else p.t().contiguous(), case["block_rows"]) for p in parts]
            out[name] = torch.stack([q for q, _ in each]).view(s["x"].shape if name == "row" else s["x"].mT.shape)
            scale = torch.stack([v for _, v in each])
            out[name + "_scale"] = scale[0] if case["batch"] == 1 else scale
        return out
    if op == "product":
        return _exact_values(s["a"], s["a_scale"], 1) @ _exact_values(s["b"], s["b_scale"], case["block_rows"]).t()
    offsets = s["offsets"].tolist()
    a = _exact_values(s["a"], s["a_scale"], 1)
    if op == "experts":
        y = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            r = slice(offsets[e], offsets[e + 1])
            y[r] = a[r] @ _exact_values(s["b"][e], s["b_scale"][e], case["block_rows"]).t()
        return y
    b = _exact_values(s["b"], s["b_scale"], 1)
    return torch.stack([a[:, offsets[e]:offsets[e + 1]] @ b[:, offsets[e]:offsets[e + 1]].t()
                        for e in range(case["experts"])])
