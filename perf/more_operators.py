"""What is measured of the operators beside the routed experts and their layer: the microscaled
4-bit quantisation and product (inference, and a training step's three products), layer norm with
its backward pass, and the whole routed layer of a few tokens.

Each case is one pass.  With `own` false, run() evaluates the formulas with elementary torch
operations in 32 bits (64 for the router's selection keys, whose order must not depend on
rounding); with `own` true it calls the library.  exact() evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
BETA, LINEAR_BETA = 4.0, 25.0

# ------------------------------------------------------------------------------------- cases


def _linear(name, T, N, K, a, act, add):
    """Inference: tokens coded as `a`, times MXFP4 weights of N rows (gate and up rows where act is set)."""
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "a": a, "act": act, "add": add}


def _train(name, T, N, K, a, x, noise):
    """A training step's three products: x's type; `a` codes the left operands; noise: the output's
    gradient is rounded stochastically."""
    return {"name": name, "op": "train", "T": T, "N": N, "K": K, "a": a, "x": x, "noise": noise}


def _norm(name, T, D, res, y, train):
    """res: type of the residual stream; y: with a block's output to add."""
    return {"name": name, "op": "norm", "T": T, "D": D, "res": res, "y": y, "train": train}


def _few(name, T, E, K, D, I, a, act, score, bias, dt):
    return {"name": name, "op": "few", "T": T, "E": E, "K": K, "D": D, "I": I, "a": a, "act": act, "score": score,
            "bias": bias, "dt": dt}


def listed():
    return [
        # the [gate|up] projection of a dense MXFP4 block for one decoded token
        _linear("mx-dec-1", 1, 7168, 3584, "fp8", "situv2", False),
        # a down projection for a serving batch, summed with what the routed experts gave
        _linear("mx-mid-200", 200, 3584, 3584, "fp4", "", True),
        # the [gate|up] projection for a prefill chunk
        _linear("mx-pre-8192", 8192, 7168, 3584, "fp4", "silu", False),
        # forward, input gradient and weight gradient of a linear layer trained in MXFP4
        _train("mx-train-4096", 4096, 3584, 3584, "fp4", "bf16", True),
        # the same for a ragged batch and widths that no block divides, fp8 on the left
        _train("mx-train-777", 777, 1000, 1790, "fp8", "f32", False),
        # layer norm of one decoded token, with the residual sum before it
        _norm("ln-dec-1", 1, 3584, "bf16", True, False),
        # of a prefill chunk
        _norm("ln-pre-8192", 8192, 3584, "bf16", True, False),
        # of a training step with an fp32 residual stream: forward, backward, weight gradients
        _norm("ln-train-4096", 4096, 3584, "f32", True, True),
        # of a small model's ragged batch, a width that no vector load divides
        _norm("ln-train-777", 777, 1790, "bf16", False, True),
        # the routed layer of one decoded token, bf16 activations
        _few("few-dec-1", 1, 896, 16, 3584, 384, "bf16", "situv2", "softmax", False, "f32"),
        # of a decode batch, fp8 activations, sigmoid scores with a selection bias
        _few("few-dec-16", 16, 896, 16, 3584, 384, "fp8", "situv2", "sigmoid", True, "f32"),
        # of a small model's three tokens
        _few("few-small-3", 3, 40, 6, 896, 256, "bf16", "silu", "softmax", False, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["linear", "linear", "train", "norm", "norm", "few", "few"])
    if kind == "linear":
        act = rng.choice(["", "", "situv2", "silu"])
        K = _log(rng, 1, 224) * 32
        N = _log(rng, 1, 224) * 32 if act else _log(rng, 17, 7168)
        T = _log(rng, 1, min(8192, max(1, 200_000_000_000 // (N * K))))
        return _linear("", T, N, K, rng.choice(["fp8", "fp4"]), act, rng.random() < 0.5)
    if kind == "train":
        N, K = _log(rng, 33, 4096), _log(rng, 33, 4096)
        T = _log(rng, 16, min(8192, max(16, 50_000_000_000 // (N * K))))
        return _train("", T, N, K, rng.choice(["fp8", "fp4"]), rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    if kind == "norm":
        T = _log(rng, 1, 16384)
        D = _log(rng, 64, min(16384, max(64, 14_000_000 // T)))
        return _norm("", T, D, rng.choice(["bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.5)
    E = _log(rng, 4, 896)
    D = 128 * _log(rng, 1, 28)
    I = 128 * _log(rng, 1, max(1, min(16, 9632 // E if D > 1792 else 16)))
    I = min(I, max(128, 1_240_000_000 // (E * D) // 128 * 128))
    K = rng.randint(1, min(E, 16))
    T = _log(rng, 1, min(16, max(1, 352_000_000 // (K * I * D))))
    return _few("", T, E, K, D, I, rng.choice(["bf16", "fp8"]), rng.choice(["situv2", "silu"]),
                rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, rng.choice(["bf16", "f32"]))


def work(case):
    c = case
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        No = N // 2 if c["act"] else N
        return {"bytes": 2 * T * K + N * K * 17 / 32 + 2 * T * No * (2 if c["add"] else 1), "flops": 2 * T * N * K}
    if c["op"] == "train":                                    # x, w, dy in; y, dx, dw out
        T, N, K = c["T"], c["N"], c["K"]
        el = 2 if c["x"] == "bf16" else 4
        return {"bytes": T * K * el + N * K * 4 + T * N * 2 * 2 + (T * N if c["noise"] else 0) + 2 * T * K + 4 * N * K,
                "flops": 6 * T * N * K}
    if c["op"] == "norm":
        T, D = c["T"], c["D"]
        r = 2 if c["res"] == "bf16" else 4
        y = 1 if c["y"] else 0
        byts = T * D * (r + 2 + y * (2 + r)) + 8 * D          # x, y in; h, n out; weight and bias
        flops = 9 * T * D
        if c["train"]:                                        # dh, dn in; dx, dy, dw, db out
            byts += T * D * (2 * r + 2 + 2 * y) + 8 * D
            flops += 16 * T * D
        return {"bytes": byts, "flops": flops}
    T, E, K, D, I = (c[k] for k in ("T", "E", "K", "D", "I"))
    experts = E * (1 - (1 - K / E) ** T)                      # different ones, as independent tokens choose them
    el = {"bf16": 2, "fp8": 33 / 32}[c["a"]]
    return {"bytes": experts * 3 * I * D * 17 / 32 + T * D * (el + 2) + T * E * (2 if c["dt"] == "bf16" else 4) + 8 * T * K,
            "flops": 6 * T * K * I * D}


# ------------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # e2m1 codes of normal weights whose blocks fill the range: a nibble for each of 256 equal shares
    share = torch.special.ndtri((torch.arange(256, device=dev) + 0.5) / 256) * 2.2
    grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=dev)
    nibble = (share[:, None] - grid).abs().argmin(1).to(torch.uint8)

    def codes(*shape):
        pick = lambda: nibble[torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8).int()]  # noqa: E731
        return pick() | (pick() << 4)

    def scales(top, *shape):
        """e8m0 bytes of 2^top, 2^(top - 1) and 2^(top - 2)"""
        return torch.randint(125 + top, 128 + top, shape, generator=g, device=dev, dtype=torch.uint8)

    c, s = case, {"case": case}
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        s["x"] = (normal(T, K) * torch.exp(0.5 * normal(1, K))).to(torch.bfloat16)
        s["w"], s["ws"] = codes(N, K // 2), scales(-round(math.log2(2 * K) / 2), N, K // 32)
        s["add"] = normal(T, N // 2 if c["act"] else N).to(torch.bfloat16) if c["add"] else None
        if own:                                               # the layout a program keeps its weights in
            import quantized_moe_expert_sort_amd as qm
            s["packed"] = qm.moe_pack_mx(s["w"], s["ws"])
            del s["w"], s["ws"]
    elif c["op"] == "train":
        T, N, K = c["T"], c["N"], c["K"]
        s["x"] = (normal(T, K) * torch.exp(0.5 * normal(1, K))).to(_TYPES[c["x"]])
        s["w"] = normal(N, K) / math.sqrt(K)                  # the optimizer's fp32 weights
        s["dy"] = (normal(T, N) * torch.exp(normal(T, 1)) / T).to(torch.bfloat16)
        s["noise"] = (torch.randint(0, 256, (T, N), generator=g, device=dev, dtype=torch.uint8) if c["noise"] else None)
    elif c["op"] == "norm":
        T, D = c["T"], c["D"]
        rows, cols = torch.exp(0.5 * normal(T, 1)), torch.exp(0.5 * normal(1, D))
        s["x"] = (4 * normal(T, D) * rows * cols + normal(1, D)).to(_TYPES[c["res"]])
        s["y"] = (normal(T, D) * cols).to(torch.bfloat16) if c["y"] else None
        s["w"], s["b"] = 1 + 0.2 * normal(D), 0.2 * normal(D)
        if c["train"]:
            s["dh"] = normal(T, D).to(_TYPES[c["res"]])
            s["dn"] = normal(T, D).to(torch.bfloat16)
    else:
        T, E, K, D, I = (c[k] for k in ("T", "E", "K", "D", "I"))
        s["logits"] = (1.5 * normal(T, E)).to(_TYPES[c["dt"]])
        s["bias"] = 0.05 * normal(E) if c["bias"] else None
        s["w1"], s["w1s"] = codes(E, 2 * I, D // 2), scales(-round(math.log2(2 * D) / 2), E, 2 * I, D // 32)
        s["w2"], s["w2s"] = codes(E, D, I // 2), scales(-round(math.log2(2 * I) / 2), E, D, I // 32)
        x = normal(T, D)
        if c["a"] == "bf16":
            s["x"], s["xs"] = x.to(torch.bfloat16), None
        else:                                                 # as the norm before the layer hands them over
            v, e = _parts(x, c["a"])
            s["x"] = v.reshape(T, D).to(torch.float8_e4m3fn).view(torch.uint8)
            s["xs"] = (e[:, :, 0] + 127).to(torch.uint8)
        if own:
            import quantized_moe_expert_sort_amd as qm
            s["w1"], s["w2"] = qm.moe_pack_w1(s["w1"]), qm.moe_pack_w2(s["w2"])
    return s


# ------------------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _betas(c):
    return dict(beta=BETA, linear_beta=LINEAR_BETA) if c["act"] == "situv2" else {}


def _own_linear(s):
    import quantized_moe_expert_sort_amd as qm
    c = s["case"]
    a = qm.moe_quant_mx(s["x"], c["a"])
    return qm.moe_gemm_mx(a.q, a.q_scale, c["a"], *s["packed"], c["N"], act=c["act"] or None, add=s["add"], **_betas(c))


def _own_train(s):
    import quantized_moe_expert_sort_amd as qm
    c, a = s["case"], s["case"]["a"]
    T, N, K = c["T"], c["N"], c["K"]
    w = qm.moe_quant_mx(s["w"], "fp4", packed=True, t_dtype="fp4", t_packed=True)
    x = qm.moe_quant_mx(s["x"], a, t_dtype="fp4", t_packed=True)
    y = qm.moe_gemm_mx(x.q, x.q_scale, a, w.q, w.q_scale, N)
    d = qm.moe_quant_mx(s["dy"], a, t_dtype=a, noise=s["noise"])
    dx = qm.moe_gemm_mx(d.q, d.q_scale, a, w.t, w.t_scale, K)
    dw = qm.moe_gemm_mx(d.t, d.t_scale, a, x.t, x.t_scale, K, out_dtype=torch.float32)
    return {"y": y, "dx": dx, "dw": dw}


def _own_norm(s):
    import quantized_moe_expert_sort_amd as qm
    r = qm.moe_layer_norm(s["x"], s["y"], w=s["w"], b=s["b"], eps=EPS, stats=s["case"]["train"])
    out = {"n": r.n}
    if s["y"] is not None:
        out["h"] = r.h
    if s["case"]["train"]:
        d = qm.moe_layer_norm_backward(s["x"], s["y"], r.stats, s["dh"], s["dn"], w=s["w"])
        out.update(dx=d.dx, dw=d.dw, db=d.db)
        if s["y"] is not None:
            out["dy"] = d.dy
    return out


def _own_few(s):
    import quantized_moe_expert_sort_amd as qm
    c = s["case"]
    r = qm.moe_routed_few(s["logits"], s["x"], s["xs"], c["a"], s["w1"], s["w1s"], s["w2"], s["w2s"], c["K"],
                          score=c["score"], bias=s["bias"], act=c["act"], **_betas(c))
    return {"out": r.out, "ids": r.ids, "w": r.w}


_OWN = {"linear": _own_linear, "train": _own_train, "norm": _own_norm, "few": _own_few}

# ------------------------------------------------------------------------------------- plain form

_FMT = {"fp8": (8, 448.0, -6, 3), "fp4": (2, 6.0, 0, 1)}      # emax, largest value, lowest exponent, mantissa bits


def _times(x, k):
    """x 2^k for whole k (torch's ldexp takes a rounded power)."""
    return x * ((k.clamp(-126, 127) + 127).int() << 23).view(torch.float32)


def _parts(x, kind, noise=None):
    """x [R, C] in fp32 -> the values of its codes in units of their block's scale [R, C / 32, 32] and
    the scales' exponents [R, C / 32, 1]; C filled up with zeros."""
    emax, top, low, mant = _FMT[kind]
    fill = -x.shape[1] % 32
    b = torch.nn.functional.pad(x, (0, fill)).reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - emax, -126).clamp(-126, 127)
    v = _times(b, -e).abs().clamp(max=top)
    step = torch.frexp(v)[1] - 1
    step = torch.where(v > 0, step, low).clamp(min=low) - mant
    t = _times(v, -step)                                  # in units of the last place
    if noise is None:
        t = torch.round(t)
    else:
        n = torch.nn.functional.pad(noise.float(), (0, fill)).reshape(b.shape)
        t = torch.floor(t + (2 * n + 1) / 512)
    return torch.copysign(_times(t, step), b), e


def _code(x, kind, noise=None):
    """The values of x's codes, in fp32 [R, C]."""
    v, e = _parts(x, kind, noise)
    return _times(v, e).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _decode(q, scale, kind="fp4"):
    """Codes [..., C] or packed pairs [..., C / 2] and e8m0 bytes [..., C / 32] -> fp32 values."""
    if kind == "fp8":
        v = q.view(torch.float8_e4m3fn).float()
    else:
        nib = torch.stack((q & 15, q >> 4), -1).flatten(-2)
        grid = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=q.device)
        v = grid[nib.int()]
    mult = _times(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * mult.unsqueeze(-1)).flatten(-2)


def _activate(c, g, u):
    if c["act"] == "silu":
        return g * torch.sigmoid(g) * u
    return BETA * torch.tanh(g / BETA) * torch.sigmoid(g) * LINEAR_BETA * torch.tanh(u / LINEAR_BETA)


def _plain_linear(s):
    c = s["case"]
    r = _code(s["x"].float(), c["a"]) @ _decode(s["w"], s["ws"]).t()
    if c["act"]:
        r = _activate(c, r[:, : c["N"] // 2], r[:, c["N"] // 2:])
    if s["add"] is not None:
        r = r + s["add"].float()
    return r.to(torch.bfloat16)


def _plain_train(s):
    a, noise = s["case"]["a"], s["noise"]
    x, w, dy = s["x"].float(), s["w"], s["dy"].float()
    y = _code(x, a) @ _code(w, "fp4").t()
    dx = _code(dy, a, noise) @ _code(w.t(), "fp4").t()
    dw = _code(dy.t(), a, None if noise is None else noise.t()) @ _code(x.t(), "fp4").t()
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw}


def _plain_norm(s):
    D, res = s["case"]["D"], s["x"].dtype
    h = s["x"].float()
    if s["y"] is not None:
        h = h + s["y"].float()
    mean = h.sum(1, keepdim=True) / D
    z = h - mean
    r = torch.rsqrt((z * z).sum(1, keepdim=True) / D + EPS)
    z = z * r
    out = {"n": (z * s["w"] + s["b"]).to(torch.bfloat16)}
    if s["y"] is not None:
        out["h"] = h.to(res)
    if s["case"]["train"]:
        dn = s["dn"].float()
        u = dn * s["w"]
        e = s["dh"].float() + r * (u - u.sum(1, keepdim=True) / D - z * ((u * z).sum(1, keepdim=True) / D))
        out.update(dx=e.to(res), dw=(dn * z).sum(0), db=dn.sum(0))
        if s["y"] is not None:
            out["dy"] = e.to(torch.bfloat16)
    return out


def _plain_few(s):
    c = s["case"]
    T, K, I = c["T"], c["K"], c["I"]
    l = s["logits"].float()
    soft = torch.exp(l - l.amax(1, keepdim=True))
    score = soft / soft.sum(1, keepdim=True) if c["score"] == "softmax" else torch.sigmoid(l)
    keys = l                                                  # the score grows with the logit
    if s["bias"] is not None:
        wide = l.double()
        wide = torch.softmax(wide, 1) if c["score"] == "softmax" else torch.sigmoid(wide)
        keys = wide + s["bias"].double()
    ids = torch.sort(keys, dim=1, descending=True, stable=True)[1][:, :K]
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    x = s["x"].float() if c["a"] == "bf16" else _decode(s["x"], s["xs"], c["a"])
    e = ids.reshape(-1)
    r = (_decode(s["w1"][e], s["w1s"][e]) @ x.repeat_interleave(K, 0).unsqueeze(2)).squeeze(2)
    m = _activate(c, r[:, :I], r[:, I:])
    if c["a"] != "bf16":
        m = _code(m, c["a"])
    o = (_decode(s["w2"][e], s["w2s"][e]) @ m.unsqueeze(2)).reshape(T, K, -1)
    return {"out": (o * w[:, :, None]).sum(1).to(torch.bfloat16), "ids": ids.int(), "w": w}


_PLAIN = {"linear": _plain_linear, "train": _plain_train, "norm": _plain_norm, "few": _plain_few}

# ------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    global own
    was, own = own, False                                     # inputs only; no weights laid out
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"linear": _exact_linear, "train": _exact_train, "norm": _exact_norm, "few": _exact_few}[case["op"]](case, s)


def _exact_code(x, kind, noise=None):
    """By the definition: blocks of 32 of a row share a power of two, floor(log2 of the largest) less the
    format's largest exponent; values between two neighbours of the grid go to the nearer, the even one of
    two as near, or up with the chance that the noise stands for."""
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    if kind == "fp8":
        pos = torch.arange(127, device=x.device, dtype=torch.uint8)
        grid = pos.view(torch.float8_e4m3fn).double()
    emax = 2 if kind == "fp4" else 8
    rows, cols = x.shape
    whole = (cols + 31) // 32 * 32
    full = torch.zeros(rows, whole, dtype=torch.float64, device=x.device)
    full[:, :cols] = x.double()
    b = full.view(rows, whole // 32, 32)
    largest = b.abs().max(2, keepdim=True).values
    unit = torch.exp2(torch.floor(torch.log2(torch.where(largest > 0, largest, torch.ones_like(largest)))) - emax)
    v = torch.minimum((b / unit).abs(), grid[-1])
    hi = torch.searchsorted(grid, v.contiguous()).clamp(1, grid.numel() - 1)
    below, above = grid[hi - 1], grid[hi]
    part = (v - below) / (above - below)
    if noise is None:
        up = (part > 0.5) | ((part == 0.5) & (hi % 2 == 0))
    else:
        n = torch.zeros(rows, whole, dtype=torch.float64, device=x.device)
        n[:, :cols] = noise.double()
        up = part + (n.view_as(b) + 0.5) / 256 >= 1
    return (torch.where(up, above, below) * b.sign() * unit).view(rows, whole)[:, :cols]


def _exact_values(q, scale):
    out = torch.empty(*q.shape, 2, dtype=torch.float64, device=q.device)
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)
    for half, code in enumerate((q % 16, q // 16)):
        out[..., half] = grid[(code % 8).int()] * (1 - 2.0 * (code // 8))
    return out.view(*q.shape[:-1], -1) * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)


def _exact_act(c, g, u):
    s = 1 / (1 + (-g).exp())
    return g * s * u if c["act"] == "silu" else BETA * (g / BETA).tanh() * s * LINEAR_BETA * (u / LINEAR_BETA).tanh()


def _exact_linear(c, s):
    r = _exact_code(s["x"], c["a"]) @ _exact_values(s["w"], s["ws"]).t()
    if c["act"]:
        r = _exact_act(c, *r.chunk(2, 1))
    return r if s["add"] is None else r + s["add"].double()


def _exact_train(c, s):
    a, n = c["a"], s["noise"]
    nt = None if n is None else n.t()
    return {"y": _exact_code(s["x"], a) @ _exact_code(s["w"], "fp4").t(),
            "dx": _exact_code(s["dy"], a, n) @ _exact_code(s["w"].t(), "fp4").t(),
            "dw": _exact_code(s["dy"].t(), a, nt) @ _exact_code(s["x"].t(), "fp4").t()}


def _exact_norm(c, s):
    leaves = {k: s[k].double().requires_grad_(True) for k in ("x", "y", "w", "b") if s[k] is not None}
    h = leaves["x"] + leaves["y"] if "y" in leaves else leaves["x"]
    n = (h - h.mean(1, keepdim=True)) / (h.var(1, correction=0, keepdim=True) + EPS).sqrt() * leaves["w"] + leaves["b"]
    out = {"n": n.detach()}
    if "y" in leaves:
        out["h"] = h.detach()
    if c["train"]:
        got = dict(zip(leaves, torch.autograd.grad((h, n), list(leaves.values()), (s["dh"].double(), s["dn"].double()))))
        out.update(dx=got["x"], dw=got["w"], db=got["b"])
        if "y" in got:
            out["dy"] = got["y"]
    return out


def _exact_few(c, s):
    T, K = c["T"], c["K"]
    l = s["logits"].double()
    sc = l.softmax(1) if c["score"] == "softmax" else 1 / (1 + (-l).exp())
    key = l if s["bias"] is None else sc + s["bias"].double()
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = sc.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    x = s["x"].double()
    if c["a"] == "fp8":
        x = s["x"].view(torch.float8_e4m3fn).double() * torch.exp2(s["xs"].double() - 127).repeat_interleave(32, 1)
    out = torch.zeros(T, c["D"], dtype=torch.float64, device=x.device)
    for t in range(T):
        g, u = (_exact_values(s["w1"][ids[t]], s["w1s"][ids[t]]) @ x[t]).chunk(2, 1)
        m = _exact_act(c, g, u)
        if c["a"] == "fp8":
            m = _exact_code(m, "fp8")
        rows = torch.matmul(_exact_values(s["w2"][ids[t]], s["w2s"][ids[t]]), m[:, :, None])
        out[t] = (w[t][:, None] * rows[:, :, 0]).sum(0)
    return {"out": out, "ids": ids.int(), "w": w}
