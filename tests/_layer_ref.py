"""Plain float64 evaluations (torch on the CPU) of the operators around the routed experts: the
block norms, the router with its losses, the 8-bit integer product.  Written from the formulas of
include/moe_mi355x.h; shares no code with the library."""
import math

import torch

MAXF = torch.finfo(torch.float32).max
HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24     # a rounding, relative to the value (HALF_F32 of fp32)


def f64(t):
    return None if t is None else t.detach().cpu().double()


def half_step(dtype):
    return HALF_BF16 if dtype == torch.bfloat16 else HALF_F32


# ------------------------------------------------------------------ block norm

def norm_forward(x, y, w_post, gate, kind, act, scale, w_pre, eps):
    """float64 (differentiable) h, n and the magnitude |x| + |scale g z| of h's terms."""
    h, mag = x, x.abs()
    if y is not None:
        z = y
        if w_post is not None:
            z = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * w_post
        if kind != "none":
            g = gate[:, None] if kind == "token" else gate
            z = z * (torch.sigmoid(g) if act == "sigmoid" else g)
        h = x + scale * z
        mag = x.abs() + (scale * z).abs()
    n = None
    if w_pre is not None:
        n = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w_pre
    return h, n, mag


def norm_backward(x, y, w_post, gate, kind, act, scale, w_pre, eps, dh, dn):
    """The gradients by the formulas, and for each the sum of the magnitudes of its terms."""
    D = x.shape[1]
    one = torch.ones(1, dtype=torch.float64)
    g = one if kind == "none" else gate[:, None] if kind == "token" else gate
    s = torch.sigmoid(g) if act == "sigmoid" else g
    slope = s * (1 - s) if act == "sigmoid" else one
    h, mag = x, x.abs()
    if y is not None:
        ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if w_post is not None else one
        w = w_post if w_post is not None else one
        yh = y * ry
        h = x + scale * s * yh * w
        mag = x.abs() + (scale * s * yh * w).abs()
    e = torch.zeros_like(x) if dh is None else dh
    me = e.abs()
    out, m = {}, {}
    if dn is not None:
        rh = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
        hh, mh = h * rh, mag * rh
        u = dn * w_pre
        e = e + rh * (u - hh * (u * hh).mean(1, keepdim=True))
        me = me + rh * (u.abs() + mh * (u.abs() * mh).mean(1, keepdim=True))
        out["dw_pre"], m["dw_pre"] = (dn * hh).sum(0), (dn.abs() * mh).sum(0)
    out["dx"], m["dx"] = e, me
    if y is not None:
        dz, mz = scale * s * e, abs(scale) * s.abs() * me
        if w_post is not None:
            out["dw_post"], m["dw_post"] = (dz * yh).sum(0), (mz * yh.abs()).sum(0)
            v, mv = dz * w, mz * w.abs()
            out["dy"] = ry * (v - yh * (v * yh).mean(1, keepdim=True))
            m["dy"] = ry * (mv + yh.abs() * (mv * yh.abs()).mean(1, keepdim=True))
        else:
            out["dy"], m["dy"] = dz, mz
        if kind != "none":
            dg, mg = scale * yh * w * e * slope, abs(scale) * (yh * w).abs() * me * slope.abs()
            red = {"channel": 0, "token": 1}.get(kind)
            out["dgate"], m["dgate"] = (dg, mg) if red is None else (dg.sum(red), mg.sum(red))
    return out, m


# ------------------------------------------------------------------ router

def masked_logits(logits):
    l = f64(logits)
    l = torch.where(l > -math.inf, l.clamp(max=MAXF), torch.full_like(l, -math.inf))   # NaN masks too
    return l + 0.0


def router_choice(logits, K, score, bias=None, valid=None):
    """ids [T, K] (-1 where nothing is left)."""
    l = masked_logits(logits)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    key = l
    if bias is not None:
        b = f64(bias)
        ok = (l > -math.inf) & (b > -math.inf)
        key = torch.where(ok, s + b.clamp(max=MAXF), torch.full_like(l, -math.inf))
    key, order = key.sort(dim=1, descending=True, stable=True)
    ids = torch.where(key[:, :K] > -math.inf, order[:, :K], -1)
    if valid is not None:
        ids = torch.where(valid.cpu().bool()[:, None], ids, -1)
    return ids.int()


def counted(logits, valid):
    ok = (masked_logits(logits) > -math.inf).any(1)
    return ok if valid is None else ok & valid.cpu().bool()


def router_outputs(l, ids, score, renorm, scale, ok, coef, z_coef):
    """(w, counts, mean_prob, loss), differentiable in l (float64, masked entries -inf) for given ids."""
    T, E = l.shape
    K = ids.shape[1]
    on = ids >= 0
    at = ids.clamp(min=0).long()
    rows = torch.where(ok[:, None], l, torch.zeros_like(l))            # uncounted rows: any finite value
    # quotients of scores as softmaxes of their logarithms: defined however negative the logits are
    lp = rows if score == "softmax" else torch.nn.functional.logsigmoid(rows)
    if renorm:
        chosen = torch.where(on, lp.gather(1, at), -math.inf)
        chosen = torch.where(on.any(1, keepdim=True), chosen, 0.0)
        v = torch.where(on, torch.softmax(chosen, 1), 0.0)
    else:
        p = torch.softmax(rows, 1) if score == "softmax" else torch.sigmoid(rows)
        v = torch.where(on, p.gather(1, at), 0.0)
    w = scale * v
    n = max(int(ok.sum()), 1)
    counts = torch.bincount(at[on], minlength=E)
    share = torch.softmax(lp, 1)
    mean = (share * ok[:, None]).sum(0) / n
    balance = coef * (counts * (E / (K * n)) * mean).sum()
    z = z_coef * (torch.logsumexp(rows, 1).square() * ok).sum() / n
    return w, counts, mean, torch.stack((balance, z))


# ------------------------------------------------------------------ 8-bit integers

def quant_i8(x):
    """(codes, scales) of float64 rows that fp32 holds: the rule in fp32 arithmetic."""
    x = x.float()
    amax = x.abs().amax(1)
    tiny = amax < 2.0 ** -100
    safe = torch.where(tiny, torch.ones_like(amax), amax)
    mul = torch.where(tiny, torch.zeros_like(amax), torch.tensor(127.0) / safe)
    q = torch.round(x * mul[:, None]).clamp(-127, 127)
    return q.to(torch.int8), torch.where(tiny, torch.zeros_like(amax), amax / torch.tensor(127.0))


def gemm_i8(a, sa, w, sw, act=None, beta=4.0, lb=25.0, add=None):
    """float64 result and the bound of its fp32 error before the last rounding: two products of
    scales and one of the sum (whose conversion to fp32 rounds too), so 4 roundings of r; the
    activations' exponentials and quotient are off by a few 2^-23 of 1 (absolute, before the factors
    beta and lb), taken as 16."""
    r = (f64(a) @ f64(w).t()) * f64(sa)[:, None] * f64(sw)
    err = 4 * HALF_F32 * r.abs()
    if act is not None:
        half = r.shape[1] // 2
        g, u = r[:, :half], r[:, half:]
        if act == "silu":
            s = torch.sigmoid(g)
            r = g * s * u
            err = 32 * HALF_F32 * (1 + g.abs()) * (g * s * u).abs()
        else:
            tg, tu, s = torch.tanh(g / beta), torch.tanh(u / lb), torch.sigmoid(g)
            r = beta * tg * s * lb * tu
            err = 32 * HALF_F32 * beta * lb * s * (tg.abs() + tu.abs() + (1 + g.abs()) * (tg * tu).abs())
    if add is not None:
        err = err + HALF_F32 * (r.abs() + f64(add).abs())
        r = r + f64(add)
    return r, err
