"""4-bit operands in 64-bit arithmetic, for the tests: codes, scales, layouts and random operands."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2M1 = torch.cat([E2M1, -E2M1])


def unpack(data):
    """Values of packed codes."""
    return E2M1[torch.stack([data & 15, data >> 4], -1).flatten(-2).long()]


def swizzle(scale):
    """[R, C] bytes -> the 128x4 layout, from its formula (R % 128 == 0, C % 4 == 0)."""
    R, C = scale.shape
    r, c = torch.meshgrid(torch.arange(R), torch.arange(C), indexing="ij")
    at = (r // 128 * (C // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
    out = torch.empty(R * C, dtype=scale.dtype)
    out[at.reshape(-1)] = scale.reshape(-1)
    return out


def scale_values(scale, block):
    """What scale bytes stand for, without the amax."""
    if block == 32:
        s = torch.ldexp(torch.ones((), dtype=torch.float64), scale.int() - 127)
        return torch.where(scale == 255, torch.nan, s)
    return scale.view(torch.float8_e4m3fn).double()


def values(data, scale, amax, block):
    """[rows, cols] values of compact scales [rows, cols / block]; amax: None, [1] or [rows]."""
    v = unpack(data) * scale_values(scale, block).repeat_interleave(block, 1)
    return v if amax is None else v * (amax.double() / 2688.0)[:, None]


def random_parts(rows, cols, block, seed, exact=False, per_row=False):
    """(codes, compact scales, amax) of a random operand.  exact: scales 1/2, 1 and 2 and an amax of 2688, so that
    every product of two such operands is a multiple of 2^-4, below 576: sums of some thousand of them are exact in
    32 bits in any order."""
    g = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8)
    shape = (rows, cols // block)
    if block == 32:
        lo, hi = (126, 129) if exact else (110, 140)
        return data, torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8), None
    if exact:
        scale = (0x30 + 8 * torch.randint(0, 3, shape, generator=g)).to(torch.uint8)
        return data, scale, torch.full((rows if per_row else 1,), 2688.0)
    scale = torch.randint(1, 127, shape, generator=g, dtype=torch.uint8)
    return data, scale, torch.rand(rows if per_row else 1, generator=g) * 7 + 0.1


def operand(parts, block, swizzled=False, device="cuda"):
    import nvfp4_block_scaled_amax_gb300 as nv
    data, scale, amax = parts
    return nv.FP4Operand(data.to(device), (swizzle(scale) if swizzled else scale).to(device),
                         None if amax is None else amax.to(device), block, swizzled)


def mx_cast(x):
    """(codes one in a byte, scale bytes) of the MXFP4 cast along the rows of x, from the definition in 64 bits."""
    rows, cols = x.shape
    v = x.double().reshape(rows, cols // 32, 32)
    amax = v.abs().amax(-1)
    amax = torch.where(v.isnan().any(-1), torch.nan, amax)
    fine = torch.isfinite(amax)
    byte = torch.frexp(torch.where(fine & (amax > 0), amax, 1.0)).exponent - 1 - 2 + 127
    byte = torch.where(amax == 0, 0, byte.clamp(min=0))
    p = v * torch.ldexp(torch.ones((), dtype=torch.float64), 127 - byte)[..., None]
    a = p.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = torch.round(a / step) * step
    code = torch.searchsorted(E2M1[:8].contiguous(), a.contiguous()).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    code = torch.where(fine[..., None], code, 0)
    return code.reshape(rows, cols).to(torch.uint8), torch.where(fine, byte, 255).to(torch.uint8)


def pack(code):
    return code[..., ::2] | (code[..., 1::2] << 4)
