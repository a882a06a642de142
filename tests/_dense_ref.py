"""Plain float64 evaluations (torch) of the operators beside the routed experts: microscaled codes and
products, layer norm.  Written from the formulas of include/moe_mi355x.h; shares no code with the
library."""
import torch

HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24     # a rounding, relative to the value


def half_step(dtype):
    return HALF_BF16 if dtype == torch.bfloat16 else HALF_F32


# ------------------------------------------------------------------ microscaled codes

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()      # 0 .. 448


def mx_codes(x, kind, noise=None):
    """(codes [R, Kp] one a byte, scale bytes [R, Kp / 32]) of rows filled up with zeros to Kp, a multiple
    of 128; on the CPU."""
    grid, emax, sign = (E2M1, 2, 8) if kind == "fp4" else (E4M3, 8, 128)
    R, C = x.shape
    kp = (C + 127) // 128 * 128
    full = torch.zeros(R, kp, dtype=torch.float64)
    full[:, :C] = x.detach().cpu().double()
    b = full.view(R, kp // 32, 32)
    bad = ~torch.isfinite(b).all(2)
    b = torch.where(bad[:, :, None], 0.0, b)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - emax, -127).clamp(-127, 127)
    v = torch.ldexp(b.abs(), -e[:, :, None]).clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
    lo = hi - 1
    part = (v - grid[lo]) / (grid[hi] - grid[lo])
    if noise is None:
        up = (part > 0.5) | ((part == 0.5) & (hi % 2 == 0))
    else:
        n = torch.zeros(R, kp, dtype=torch.float64)
        n[:, :C] = noise.cpu().double()
        up = part + (2 * n.view_as(b) + 1) / 512 >= 1
    code = torch.where(up, hi, lo) + sign * torch.signbit(b)
    code = torch.where(bad[:, :, None], 0, code)
    return code.view(R, kp).to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def pairs(codes):
    """fp4 codes, one a byte, -> two a byte, the even column in the low nibble."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpairs(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(1)


def mx_values(codes, scale, kind):
    """float64 values of codes (one a byte) and scale bytes, NaN where the byte is 255."""
    if kind == "fp4":
        v = E2M1.to(codes.device)[(codes & 7).long()] * (1 - 2 * (codes >> 3).double())
    else:
        v = codes.view(torch.float8_e4m3fn).double()
    m = torch.exp2(scale.double() - 127).masked_fill(scale == 255, float("nan"))
    return v * m.repeat_interleave(32, 1)


def mx_packed(q, scale):
    """fp4x2 codes [N, Kp / 2] and scales [N, Kp / 32] -> the packed layout, by its definition."""
    N, half = q.shape
    n16 = (N + 15) // 16 * 16
    qf = torch.zeros(n16, half, dtype=torch.uint8)
    qf[:N] = q
    sf = torch.zeros(n16, scale.shape[1], dtype=torch.uint8)
    sf[:N] = scale
    blocks = qf.view(n16 // 16, 16, half // 64, 4, 16)          # f, r, s, g, b
    scales = sf.view(n16 // 16, 16, half // 64, 4)              # f, r, s, g
    return (blocks.permute(0, 2, 3, 1, 4).reshape(n16 // 16, half // 64, 1024),
            scales.permute(0, 2, 1, 3).reshape(n16 // 16, half // 64, 64))


def activated(r, act, beta=4.0, lb=25.0):
    g, u = r.chunk(2, 1)
    s = torch.sigmoid(g)
    return g * s * u if act == "silu" else beta * torch.tanh(g / beta) * s * lb * torch.tanh(u / lb)


# ------------------------------------------------------------------ layer norm

def layer_norm(x, y, w, b, eps):
    """float64 (differentiable) h, n."""
    h = x if y is None else x + y
    z = (h - h.mean(1, keepdim=True)) / torch.sqrt(h.var(1, correction=0, keepdim=True) + eps)
    n = z if w is None else z * w
    return h, n if b is None else n + b


def layer_norm_parts(h, eps):
    """(mean, rstd, z, bound of z's fp32 error).  The bound: h and the mean are rounded once each and so
    is their difference (4 steps of |h| + |m|, relative to the deviation); the sums of deviations and of
    their squares have at most 32 roundings each (16 in a lane, 10 across lanes and waves, products), the
    mean deviation is at most 1, half of the squares' error reaches 1 / sqrt, whose own steps are 4 more."""
    m = h.mean(1, keepdim=True)
    r = 1 / torch.sqrt(h.var(1, correction=0, keepdim=True) + eps)
    z = (h - m) * r
    per_row = ((h.abs() + m.abs()) * r).amax(1, keepdim=True)
    return m, r, z, HALF_F32 * (4 * (h.abs() + m.abs()) * r + 32 + (20 + 4 * per_row) * z.abs())
