"""What is measured of the operators around the routed experts of one MoE layer: the norms before
and after a block (with gate and residual scale), the router with its balance loss, and the 8-bit
integer product of the shared expert.

Each case is one pass through an operator.  With `own` false, run() evaluates the operator's
formula with elementary torch operations in 32 bits (64 for the router's selection keys, whose
order must not depend on rounding); with `own` true it calls the library.  exact() evaluates the
definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
BETA, LINEAR_BETA = 4.0, 25.0

# ------------------------------------------------------------------------------------- cases


def _norm(name, T, D, res, gate, gate_act, q, train, scale=1.0):
    """res: type of the residual stream; gate: none | channel | token | element; q: type of the
    coded output ("" for none)."""
    return {"name": name, "op": "norm", "T": T, "D": D, "res": res, "gate": gate, "gate_act": gate_act,
            "q": q, "train": train, "scale": scale}


def _router(name, T, E, K, dt, score, renorm, bias, masked, train):
    return {"name": name, "op": "router", "T": T, "E": E, "K": K, "dt": dt, "score": score, "renorm": renorm,
            "bias": bias, "masked": masked, "train": train}


def _gemm(name, T, N, K, act, add):
    """N: weight rows (gate and up rows where act is set)."""
    return {"name": name, "op": "gemm", "T": T, "N": N, "K": K, "act": act, "add": add}


def listed():
    return [
        # one decoded token between two blocks: the norm after attention, the residual sum, the norm
        # before the MoE block, coded for the int8 shared expert (and in bf16 for the router)
        _norm("norm-dec-1", 1, 3584, "bf16", "none", "none", "i8", False),
        # a prefill chunk entering the fp8 routed experts, behind a block gated per token
        _norm("norm-pre-8192", 8192, 3584, "bf16", "token", "sigmoid", "fp8", False, 0.5),
        # a training step's norm pair with a learnt scale per channel and an fp32 residual stream
        _norm("norm-train-4096", 4096, 3584, "f32", "channel", "none", "", True),
        # a small model's ragged batch, a width that no vector load divides, gated per element
        _norm("norm-train-777", 777, 1790, "bf16", "element", "sigmoid", "", True, 0.25),
        # a decode batch routed with sigmoid scores and a selection bias per expert
        _router("router-dec-16", 16, 896, 16, "f32", "sigmoid", True, True, False, False),
        # a prefill chunk routed by softmax over bf16 logits (many exact ties)
        _router("router-pre-16384", 16384, 896, 16, "bf16", "softmax", True, False, False, False),
        # a training step's routing: choice, weights, balance and z loss, and the logits' gradient
        _router("balance-train-8192", 8192, 896, 16, "f32", "softmax", True, False, False, True),
        # the same for a padded ragged batch of a smaller model with sigmoid scores and masked experts
        _router("balance-train-1501", 1501, 112, 6, "bf16", "sigmoid", True, True, True, True),
        # the shared expert's [gate|up] product for one token
        _gemm("gemm-dec-1", 1, 7168, 3584, "situv2", False),
        # its down product for a small serving batch, summed with the routed experts' output
        _gemm("gemm-mid-200", 200, 3584, 3584, "", True),
        # its [gate|up] product for a prefill chunk
        _gemm("gemm-pre-8192", 8192, 7168, 3584, "situv2", False),
        # a ragged chunk through a projection whose sizes no tile divides
        _gemm("gemm-odd-1111", 1111, 1000, 1456, "", False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["norm", "norm", "router", "router", "gemm", "gemm"])
    if kind == "norm":
        q = rng.choice(["", "", "fp8", "fp4", "i8"])
        T = _log(rng, 1, 16384)
        D = _log(rng, 64, min(16384, max(64, 14_000_000 // T)))
        D = max(32, D // 32 * 32) if q else D
        gate = rng.choice(["none", "channel", "token", "element"])
        return _norm("", T, D, rng.choice(["bf16", "f32"]), gate,
                     rng.choice(["none", "sigmoid"]) if gate != "none" else "none", q, rng.random() < 0.5,
                     rng.choice([1.0, 0.5, 0.22]))
    if kind == "router":
        train = rng.random() < 0.5
        E = _log(rng, 8, 2048)
        K = rng.randint(1, min(E, 32))
        T = _log(rng, 1, min(16384, 7_000_000 // E))
        return _router("", T, E, K, rng.choice(["bf16", "f32"]), rng.choice(["softmax", "sigmoid"]),
                       rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.3, train)
    act = rng.choice(["", "", "situv2", "silu"])
    K = _log(rng, 16, 450) * 16
    N = _log(rng, 4, 224) * 32 if act else _log(rng, 65, 7168)
    T = _log(rng, 1, min(8192, max(1, 200_000_000_000 // (N * K))))
    return _gemm("", T, N, K, act, rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "norm":
        T, D = c["T"], c["D"]
        r = 2 if c["res"] == "bf16" else 4
        gate = {"none": 0, "channel": 4 * D, "token": 4 * T, "element": 2 * T * D}[c["gate"]]
        q = {"": 0, "fp8": T * D + T * D / 32, "fp4": T * D / 2 + T * D / 32, "i8": T * D + 4 * T}[c["q"]]
        byts = T * D * (r + 2 + r + 2) + gate + q + 8 * D       # x, y in; h, n out; codes; two weights
        flops = 12 * T * D
        if c["train"]:                                          # dh, dn in; dx, dy and the small gradients out
            byts += T * D * (r + 2 + r + 2) + gate + 8 * D
            flops += 30 * T * D
        return {"bytes": byts, "flops": flops}
    if c["op"] == "router":
        T, E, K = c["T"], c["E"], c["K"]
        el = 2 if c["dt"] == "bf16" else 4
        byts = T * E * el + 8 * T * K + (T if c["masked"] else 0) + (4 * E if c["bias"] else 0)
        flops = 8 * T * E
        if c["train"]:                                          # the gradient out, the weights' gradient in
            byts += T * E * el + 4 * T * K + 8 * E
            flops += 8 * T * E
        return {"bytes": byts, "flops": flops}
    T, N, K = c["T"], c["N"], c["K"]
    No = N // 2 if c["act"] else N
    return {"bytes": T * K + N * K + 4 * T + 4 * N + 2 * T * No * (2 if c["add"] else 1), "flops": 2 * T * N * K}


# ------------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    c, s = case, {"case": case}
    if c["op"] == "norm":
        T, D = c["T"], c["D"]
        # rows of different sizes, a few channels much larger than the others, as in a residual stream
        rows, cols = torch.exp(0.5 * normal(T, 1)), torch.exp(0.5 * normal(1, D))
        s["x"] = (4 * normal(T, D) * rows * cols).to(_TYPES[c["res"]])
        s["y"] = (normal(T, D) * cols).to(torch.bfloat16)
        s["w_post"], s["w_pre"] = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D)
        shape = {"none": None, "channel": (D,), "token": (T,), "element": (T, D)}[c["gate"]]
        s["gate"] = None if shape is None else normal(*shape).to(torch.bfloat16 if c["gate"] == "element" else torch.float32)
        if c["train"]:
            s["dh"] = normal(T, D).to(_TYPES[c["res"]])
            s["dn"] = normal(T, D).to(torch.bfloat16)
    elif c["op"] == "router":
        T, E, K = c["T"], c["E"], c["K"]
        # logits with a prior of the expert's rank, as a trained router has
        prior = -0.5 * torch.log(1 + torch.randperm(E, generator=g, device=dev).float())
        logits = 1.5 * normal(T, E) + prior
        if c["masked"]:                                       # experts that are switched off, and padding
            off = torch.rand(E, generator=g, device=dev) < 0.1
            off[: min(E, 2 * K)] = False
            logits = logits.masked_fill(off, -math.inf)
        s["logits"] = logits.to(_TYPES[c["dt"]])
        s["bias"] = 0.05 * normal(E) if c["bias"] else None
        s["valid"] = (torch.rand(T, generator=g, device=dev) < 0.8) if c["masked"] else None
        if c["train"]:
            s["dw"] = normal(T, K)
            s["dloss"] = torch.rand(2, generator=g, device=dev) + 0.5
    else:
        T, N, K = c["T"], c["N"], c["K"]
        No = N // 2 if c["act"] else N
        # codes of normal activations and weights, each row filling the range
        s["a"] = (32 * normal(T, K)).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = (32 * normal(N, K)).round_().clamp_(-127, 127).to(torch.int8)
        s["sa"] = (0.5 + torch.rand(T, generator=g, device=dev)) / 32
        s["sw"] = (0.5 + torch.rand(N, generator=g, device=dev)) / (32 * math.sqrt(K))
        s["add"] = normal(T, No).to(torch.bfloat16) if c["add"] else None
        if own:                                               # the layout a program keeps its weights in
            import quantized_moe_expert_sort_amd as qm
            s["packed"] = qm.moe_pack_i8(s["w"])
            del s["w"]
    return s


COEF, Z_COEF = 0.01, 0.001

# ------------------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _own_norm(s):
    import quantized_moe_expert_sort_amd as qm
    c = s["case"]
    r = qm.moe_block_norm(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], gate_kind=c["gate"],
                          gate_act=c["gate_act"], scale=c["scale"], w_pre=s["w_pre"], eps=EPS,
                          q_dtype=c["q"] or None, stats=c["train"])
    out = {"h": r.h, "n": r.n}
    if c["q"]:
        out["q"] = _values(r.q, r.q_scale, c["q"])
    if c["train"]:
        b = qm.moe_block_norm_backward(s["x"], s["y"], r.rstd, s["dh"], s["dn"], w_post=s["w_post"], gate=s["gate"],
                                       gate_kind=c["gate"], gate_act=c["gate_act"], scale=c["scale"], w_pre=s["w_pre"])
        out.update(dx=b.dx, dy=b.dy, dw_post=b.dw_post, dw_pre=b.dw_pre)
        if s["gate"] is not None:
            out["dgate"] = b.dgate
    return out


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(q, scale, kind):
    """The values that codes and scales stand for, in bf16."""
    if kind == "i8":
        return (q.float() * scale[:, None]).to(torch.bfloat16)
    T = q.shape[0]
    if kind == "fp8":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        nib = torch.stack((q & 15, q >> 4), -1).reshape(T, -1)
        grid = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=q.device)
        v = grid[nib.long()]
    mult = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    return (v.reshape(T, -1, 32) * mult[:, :, None]).reshape(T, -1).to(torch.bfloat16)


def _own_router(s):
    import quantized_moe_expert_sort_amd as qm
    c = s["case"]
    kw = dict(score=c["score"], renorm=c["renorm"], valid=s["valid"])
    if not c["train"]:
        r = qm.moe_router(s["logits"], c["K"], bias=s["bias"], **kw)
        return {"ids": r.ids, "w": r.w}
    r = qm.moe_router(s["logits"], c["K"], bias=s["bias"], balance=(COEF, Z_COEF), **kw)
    d = qm.moe_router_backward(s["logits"], r, s["dw"], d_loss=s["dloss"], **kw)
    return {"ids": r.ids, "w": r.w, "counts": r.balance.counts, "mean_prob": r.balance.mean_prob,
            "loss": r.balance.loss, "dlogits": d}


def _own_gemm(s):
    import quantized_moe_expert_sort_amd as qm
    c = s["case"]
    kw = dict(beta=BETA, linear_beta=LINEAR_BETA) if c["act"] == "situv2" else {}
    return qm.moe_gemm_i8(s["a"], s["sa"], s["packed"], s["sw"], act=c["act"] or None, add=s["add"], **kw)


_OWN = {"norm": _own_norm, "router": _own_router, "gemm": _own_gemm}

# ------------------------------------------------------------------------------------- plain form


def _code(n, kind):
    """n in fp32 -> the values of its codes, in bf16."""
    if kind == "i8":
        amax = n.abs().amax(1, keepdim=True)
        q = torch.round(n * torch.where(amax > 0, 127 / amax, 0))
        return (q * (amax / 127)).to(torch.bfloat16)
    emax, top = (8, 448.0) if kind == "fp8" else (2, 6.0)
    b = n.reshape(n.shape[0], -1, 32)
    e = torch.frexp(b.abs().amax(2, keepdim=True))[1] - 1 - emax       # floor(log2 amax) - emax
    v = torch.ldexp(b, -e).clamp(-top, top)
    if kind == "fp8":
        r = v.to(torch.float8_e4m3fn).float()
    else:                                                              # steps of 1/2 below 2, 1 below 4, then 2
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        r = torch.round(v / step) * step
    return torch.ldexp(r, e).reshape(n.shape).to(torch.bfloat16)


def _plain_norm(s):
    c, D = s["case"], s["case"]["D"]
    x, y, scale = s["x"].float(), s["y"].float(), c["scale"]
    ry = torch.rsqrt((y * y).sum(1, keepdim=True) / D + EPS)
    yh = y * ry
    z = yh * s["w_post"]
    gate = s["gate"]
    if gate is not None:
        gate = gate.float()[:, None] if c["gate"] == "token" else gate.float()
        g = torch.sigmoid(gate) if c["gate_act"] == "sigmoid" else gate
    else:
        g = 1.0
    h = x + scale * g * z
    rh = torch.rsqrt((h * h).sum(1, keepdim=True) / D + EPS)
    hh = h * rh
    n = hh * s["w_pre"]
    out = {"h": h.to(s["x"].dtype), "n": n.to(torch.bfloat16)}
    if c["q"]:
        out["q"] = _code(n, c["q"])
    if c["train"]:
        dn = s["dn"].float()
        u = dn * s["w_pre"]
        e = s["dh"].float() + rh * (u - hh * ((u * hh).sum(1, keepdim=True) / D))
        dz = scale * g * e
        v = dz * s["w_post"]
        dy = ry * (v - yh * ((v * yh).sum(1, keepdim=True) / D))
        out.update(dx=e.to(s["x"].dtype), dy=dy.to(torch.bfloat16), dw_post=(dz * yh).sum(0), dw_pre=(dn * hh).sum(0))
        if gate is not None:
            dg = scale * z * e
            if c["gate_act"] == "sigmoid":
                dg = dg * (g * (1 - g))
            out["dgate"] = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1),
                            "element": lambda: dg.to(torch.bfloat16)}[c["gate"]]()
    return out


def _choose(keys, K):
    """The K largest keys of each row, ties to the lowest index; -1 where the row has no more."""
    v, i = torch.sort(keys, dim=1, descending=True, stable=True)
    return torch.where(v[:, :K] > -math.inf, i[:, :K], -1)


def _plain_router(s):
    c = s["case"]
    l = s["logits"].float()
    T, E = l.shape
    K, valid = c["K"], s["valid"]
    m = l.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(l - m).sum(1, keepdim=True))
    soft = torch.exp(l - lse)
    sig = torch.sigmoid(l)
    score = soft if c["score"] == "softmax" else sig
    if s["bias"] is None:
        keys = l                                             # the score grows with the logit
    else:
        wide = l.double()
        wide = torch.exp(wide - torch.logsumexp(wide, 1, keepdim=True)) if c["score"] == "softmax" else torch.sigmoid(wide)
        keys = torch.where(l > -math.inf, wide + s["bias"].double(), -math.inf)
    ids = _choose(keys, K)
    if valid is not None:
        ids = torch.where(valid[:, None], ids, -1)
    on = ids >= 0
    at = ids.clamp(min=0)
    v = torch.where(on, score.gather(1, at), 0.0)
    total = v.sum(1, keepdim=True)
    w = torch.where(total > 0, v / total, 0.0) if c["renorm"] else v
    out = {"ids": ids.int(), "w": w}
    if c["train"]:
        ok = torch.ones(T, 1, device=l.device) if valid is None else valid.float()[:, None]
        Tv = ok.sum().clamp(min=1)
        counts = torch.zeros(E, device=l.device).index_add_(0, at.reshape(-1), on.float().reshape(-1))
        S = sig.sum(1, keepdim=True)
        p = soft if c["score"] == "softmax" else sig / S
        P = (p * ok).sum(0) / Tv
        f = counts * (E / K) / Tv
        loss = torch.stack((COEF * (f * P).sum(), Z_COEF * (lse * lse * ok).sum() / Tv))
        db, dz = s["dloss"][0], s["dloss"][1]
        a = db * COEF * f / Tv
        inner = a - (a * p).sum(1, keepdim=True)
        d = p * inner if c["score"] == "softmax" else sig * (1 - sig) * inner / S
        d = (d + (dz * 2 * Z_COEF / Tv) * lse * soft) * ok
        dw = torch.where(on, s["dw"], 0.0)
        if c["renorm"]:
            dv = torch.where(total > 0, (dw - (dw * w).sum(1, keepdim=True)) / total, 0.0)
        else:
            dv = dw
        if c["score"] == "softmax":
            t = torch.where(on, v * dv, 0.0)
            d = d.scatter_add(1, at, t) - soft * t.sum(1, keepdim=True)
        else:
            d = d.scatter_add(1, at, torch.where(on, dv * v * (1 - v), 0.0))
        out.update(counts=counts.int(), mean_prob=P, loss=loss, dlogits=d.to(s["logits"].dtype))
    return out


def _plain_gemm(s):
    c = s["case"]
    r = (s["a"].float() @ s["w"].float().t()) * s["sa"][:, None] * s["sw"]
    if c["act"]:
        g, u = r[:, : c["N"] // 2], r[:, c["N"] // 2:]
        if c["act"] == "silu":
            r = g * torch.sigmoid(g) * u
        else:
            r = BETA * torch.tanh(g / BETA) * torch.sigmoid(g) * LINEAR_BETA * torch.tanh(u / LINEAR_BETA)
    if s["add"] is not None:
        r = r + s["add"].float()
    return r.to(torch.bfloat16)


_PLAIN = {"norm": _plain_norm, "router": _plain_router, "gemm": _plain_gemm}

# ------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    global own
    was, own = own, False                                     # inputs only; no weights laid out
    try:
        s = prepare(case, seed)
    finally:
        own = was
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return {"norm": _exact_norm, "router": _exact_router, "gemm": _exact_gemm}[case["op"]](case, d)


def _exact_code(n, kind):
    if kind == "i8":
        step = n.abs().max(1, keepdim=True).values / 127
        return torch.round(n / step) * step
    emax, mant, low, top = (8, 3, -6, 448.0) if kind == "fp8" else (2, 1, 0, 6.0)
    b = n.unflatten(1, (-1, 32))
    unit = torch.exp2(torch.floor(torch.log2(b.abs().max(2, keepdim=True).values)) - emax)
    v = b / unit
    step = torch.exp2(torch.floor(torch.log2(v.abs())).clamp(min=low) - mant)
    return ((torch.round(v / step) * step).clamp(-top, top) * unit).flatten(1)


def _exact_norm(c, s):
    x, y, wo, wi, k = s["x"], s["y"], s["w_post"], s["w_pre"], c["scale"]
    leaves = [t.requires_grad_(True) for t in (x, y, wo, wi) + (() if s["gate"] is None else (s["gate"],))]
    z = y / (y.square().mean(1, keepdim=True) + EPS).sqrt() * wo
    if s["gate"] is not None:
        g = s["gate"].unsqueeze(1) if c["gate"] == "token" else s["gate"]
        z = z * (1 / (1 + (-g).exp()) if c["gate_act"] == "sigmoid" else g)
    h = x + k * z
    n = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * wi
    out = {"h": h.detach(), "n": n.detach()}
    if c["q"]:
        out["q"] = _exact_code(n.detach(), c["q"])
    if c["train"]:
        got = torch.autograd.grad((h, n), leaves, (s["dh"], s["dn"]))
        out.update(zip(("dx", "dy", "dw_post", "dw_pre", "dgate"), got))
    return out


def _exact_router(c, s):
    l, K, E = s["logits"].requires_grad_(True), c["K"], c["E"]
    kept = torch.ones_like(l[:, 0], dtype=torch.bool) if s["valid"] is None else s["valid"]
    with torch.no_grad():
        sc = l.softmax(1) if c["score"] == "softmax" else l.sigmoid()
        key = l if s["bias"] is None else (sc + s["bias"]).masked_fill(l == -math.inf, -math.inf)
        key, order = key.sort(dim=1, descending=True, stable=True)
        ids = order[:, :K].masked_fill((key[:, :K] == -math.inf) | ~kept[:, None], -1)
    sc = l.softmax(1) if c["score"] == "softmax" else l.sigmoid()       # its gradient is 0 at -inf
    picked = sc.gather(1, ids.clamp(min=0)) * (ids >= 0)
    w = picked
    if c["renorm"]:
        w = picked / picked.sum(1, keepdim=True).clamp(min=1e-300)
    out = {"ids": ids.int(), "w": w.detach()}
    if c["train"]:
        n = kept.sum().clamp(min=1)
        counts = torch.bincount(ids[ids >= 0].long(), minlength=E)
        p = sc / sc.sum(1, keepdim=True)
        P = p[kept].sum(0) / n
        balance = COEF * (counts * E / (K * n) * P).sum()
        z = Z_COEF * l[kept].logsumexp(1).square().sum() / n
        total = (w * s["dw"]).sum() + balance * s["dloss"][0] + z * s["dloss"][1]
        grad, = torch.autograd.grad(total, l)
        out.update(counts=counts.int(), mean_prob=P.detach(), loss=torch.stack((balance, z)).detach(), dlogits=grad)
    return out


def _exact_gemm(c, s):
    r = (s["a"].double() * s["sa"][:, None]) @ (s["w"].double() * s["sw"][:, None]).t()
    if c["act"]:
        g, u = r.chunk(2, 1)
        gated = g / (1 + (-g).exp())
        r = gated * u if c["act"] == "silu" else BETA * (g / BETA).tanh() / (1 + (-g).exp()) * LINEAR_BETA * (u / LINEAR_BETA).tanh()
    return r if s["add"] is None else r + s["add"]
