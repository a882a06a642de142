"""moe_block_norm and its backward pass against the formulas in float64, row by row and element by
element, with bounds counted from the roundings: fp32 arithmetic is taken as 64 roundings (2^-24
each) of the sum of the magnitudes of a result's terms (the sums over up to 16384 elements go
through at most 16 + 6 + 4 adds per lane and tree, the reciprocal root and the sigmoid are off by
one or two units in the last place), and each output is rounded once to its type."""
import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm
from oracle import mx_formats as mx

pytestmark = pytest.mark.gpu
ARITH = 64 * ref.HALF_F32


def make(T, D, x_dt=torch.bfloat16, kind="none", act="none", post=True, pre=True, y=True, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + D)
    n = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    c = {"x": (3 * n(T, D)).to(x_dt), "y": n(T, D).to(torch.bfloat16) if y else None,
         "w_post": 1 + 0.3 * n(D) if post else None, "w_pre": 1 + 0.3 * n(D) if pre else None}
    shape = {"none": None, "channel": (D,), "token": (T,), "element": (T, D)}[kind]
    c["gate"] = None if shape is None else n(*shape).to(torch.bfloat16 if kind == "element" else torch.float32)
    c["dh"], c["dn"] = n(T, D).to(x_dt), n(T, D).to(torch.bfloat16)
    return c


def gpu(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def close(got, want, mag, extra=0.0):
    got, tol = ref.f64(got), ref.half_step(got.dtype) * want.abs() + ARITH * mag + extra
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))


def check(T, D, x_dt=torch.bfloat16, kind="none", act="none", post=True, pre=True, y=True, scale=0.7, eps=1e-5,
          dh=True, dn=True, seed=0, shift=0):
    c = make(T, D, x_dt, kind, act, post, pre, y, seed)
    d = gpu(c)
    if shift:                                                  # storage that no 16-byte load may touch
        d = {k: None if v is None else torch.cat((v.new_zeros(shift), v.flatten()))[shift:].view(v.shape) for k, v in d.items()}
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_kind=kind, gate_act=act, scale=scale, w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], eps=eps, stats=True, **kw)
    w = {k: ref.f64(v) for k, v in c.items()}
    h, n, mag = ref.norm_forward(w["x"], w["y"], w["w_post"], w["gate"], kind, act, scale, w["w_pre"], eps)
    if y:
        assert r.h.dtype == x_dt
        close(r.h, h, mag)
    else:
        assert r.h is None
    if pre:
        rh = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
        # h's own error, and what it does to the row's norm
        row = rh * mag.square().mean(1, keepdim=True).sqrt()
        close(r.n, n, (mag * rh + h.abs() * rh * row) * w["w_pre"].abs())
    if not (dh or dn) or (dn and not pre):
        return
    b = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"] if dh else None, d["dn"] if dn else None, **kw)
    want, m = ref.norm_backward(w["x"], w["y"], w["w_post"], w["gate"], kind, act, scale, w["w_pre"], eps,
                                w["dh"] if dh else None, w["dn"] if dn else None)
    for k in b._fields:
        got = getattr(b, k)
        assert (got is None) == (k not in want), k
        if got is not None:
            # the mean over the row takes part with errors of its own: three times the magnitudes
            close(got, want[k], 3 * m[k], 1e-30)
    return d, r, b


@pytest.mark.parametrize("D", [1, 2, 7, 8, 63, 64, 100, 511, 512, 520, 1000, 1790, 3584, 4097, 8192, 8200, 12289, 16384])
def test_widths(D):
    check(3, D, kind="channel")
    check(2, D, torch.float32, kind="token", act="sigmoid")


@pytest.mark.parametrize("T", [1, 2, 4, 5, 63, 511, 513, 2049])
def test_row_counts(T):
    check(T, 256, kind="element", act="sigmoid")
    check(T, 1032, torch.float32, kind="channel", act="sigmoid")
    check(T, 97, kind="token")


@pytest.mark.parametrize("x_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,act", [("none", "none"), ("channel", "none"), ("channel", "sigmoid"), ("token", "none"),
                                      ("token", "sigmoid"), ("element", "none"), ("element", "sigmoid")])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_combinations(x_dt, kind, act, post, pre):
    check(6, 776, x_dt, kind, act, post, pre, dn=pre)
    check(6, 333, x_dt, kind, act, post, pre, dn=pre, seed=1)


@pytest.mark.parametrize("D", [9, 10, 11, 12, 13, 14, 15, 505, 513, 519, 1023, 4095, 8185, 8191, 8193, 8199, 16383])
@pytest.mark.parametrize("kind", ["channel", "element"])
def test_every_length_of_a_rows_last_piece(D, kind):
    check(5, D, kind=kind, act="sigmoid")
    check(5, D, torch.float32, kind=kind, shift=1)


@pytest.mark.parametrize("x_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(5, 11), (3, 517), (4, 5127), (2, 9001)])
def test_in_place_with_a_short_last_piece(T, D, x_dt):
    # the last elements of a row are read together with ones that other lanes store to
    d = gpu(make(T, D, x_dt, "element", "sigmoid", seed=4))
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_kind="element", gate_act="sigmoid", scale=0.5, w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], **kw)
    buf = torch.full((T + 2, D), 7.0, dtype=x_dt, device="cuda")
    for _ in range(5):
        buf[1:-1].copy_(d["x"])
        q = qm.moe_block_norm(buf[1:-1], d["y"], h=buf[1:-1], **kw)
        assert torch.equal(q.h, r.h) and torch.equal(q.n, r.n)
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()


@pytest.mark.parametrize("dh,dn", [(True, False), (False, True)])
def test_one_gradient_only(dh, dn):
    check(9, 640, kind="channel", dh=dh, dn=dn)
    check(9, 640, torch.float32, y=False, post=False, dh=dh, dn=dn)


def test_pointers_that_no_wide_load_may_read():
    check(5, 512, kind="element", shift=1)
    check(5, 512, torch.float32, kind="channel", shift=3)


def test_gradients_against_differences():
    # <gradient, direction> against the central difference of the float64 forward pass; the step
    # of 1e-4 leaves an error of about 1e-8 of the third derivative
    T, D, scale, eps = 5, 96, 0.6, 1e-4
    for kind, act in (("channel", "sigmoid"), ("token", "none"), ("element", "sigmoid")):
        c = make(T, D, torch.float32, kind, act, seed=4)
        d, r, b = check(T, D, torch.float32, kind, act, scale=scale, eps=eps, seed=4)
        w = {k: ref.f64(v) for k, v in c.items()}
        g = torch.Generator().manual_seed(5)
        for name, grad in (("x", b.dx), ("y", b.dy), ("gate", b.dgate), ("w_post", b.dw_post), ("w_pre", b.dw_pre)):
            v = torch.randn(w[name].shape, generator=g, dtype=torch.float64)

            def value(s):
                a = dict(w, **{name: w[name] + s * v})
                h, n, _ = ref.norm_forward(a["x"], a["y"], a["w_post"], a["gate"], kind, act, scale, a["w_pre"], eps)
                return float((h * w["dh"]).sum() + (n * w["dn"]).sum())
            want = (value(1e-4) - value(-1e-4)) / 2e-4
            got = float((ref.f64(grad) * v).sum())
            size = float((ref.f64(grad) * v).abs().sum())
            assert abs(got - want) <= size * (ref.half_step(grad.dtype) + 1e-5) + 1e-6, (kind, name, got, want)


def test_in_place_and_repeatable():
    c = gpu(make(40, 1000, kind="channel"))
    kw = dict(w_post=c["w_post"], gate=c["gate"], gate_kind="channel", w_pre=c["w_pre"], stats=True)
    a = qm.moe_block_norm(c["x"], c["y"], **kw)
    x = c["x"].clone()
    b = qm.moe_block_norm(x, c["y"], h=x, **kw)
    assert torch.equal(a.h, x) and torch.equal(a.n, b.n) and torch.equal(a.rstd, b.rstd)
    del kw["stats"]
    g1 = qm.moe_block_norm_backward(c["x"], c["y"], a.rstd, c["dh"], c["dn"], **kw)
    g2 = qm.moe_block_norm_backward(c["x"], c["y"], a.rstd, c["dh"], c["dn"], **kw)
    assert all(torch.equal(u, v) for u, v in zip(g1, g2))


def test_rows_with_infinity_or_nan_stay_to_themselves():
    c = make(6, 512, kind="token")
    c["x"][1, 5], c["y"][3, 7] = float("inf"), float("nan")
    d = gpu(c)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_kind="token", w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], q_dtype="i8", **kw)
    clean = {k: v for k, v in c.items()}
    clean["x"], clean["y"] = c["x"].clone(), c["y"].clone()
    clean["x"][1, 5], clean["y"][3, 7] = 0.0, 0.0
    e = gpu(clean)
    s = qm.moe_block_norm(e["x"], e["y"], q_dtype="i8", **kw)
    keep = [0, 2, 4, 5]
    assert torch.equal(r.n[keep], s.n[keep]) and torch.equal(r.q[keep], s.q[keep])
    assert torch.isnan(r.n[1]).any() and torch.isnan(r.n[3]).all()
    assert torch.isnan(r.q_scale[[1, 3]]).all() and (r.q[[1, 3]] == 0).all()


@pytest.mark.parametrize("T,D", [(7, 11), (600, 515), (3, 5127), (300, 8200)])
def test_backward_over_its_own_gradient(T, D, monkeypatch):
    # dx may be dh
    d = gpu(make(T, D, kind="channel", act="sigmoid", seed=6))
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_kind="channel", gate_act="sigmoid", w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], stats=True, **kw)
    b = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"], d["dn"], **kw)
    call = qm._call

    def over_dh(name, index, p, g, *rest):
        g.dx = g.dh
        return call(name, index, p, g, *rest)
    monkeypatch.setattr(qm, "_call", over_dh)
    dh = d["dh"].clone()
    o = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, dh, d["dn"], **kw)
    assert torch.equal(dh, b.dx)
    for got, want in zip(o[1:], b[1:]):
        assert torch.equal(got, want)


@pytest.mark.parametrize("D", [13, 515, 8195])
def test_the_end_of_a_row_does_not_see_the_next(D):
    c = make(4, D, kind="element", act="sigmoid", seed=5)
    for k in ("x", "y", "gate", "dh", "dn"):
        c[k][1] = c[k][3] = float("nan")
    d = gpu(c)
    kw = dict(w_post=d["w_post"], gate_kind="element", gate_act="sigmoid", w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], gate=d["gate"], stats=True, **kw)
    b = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"], d["dn"], gate=d["gate"], **kw)
    one = {k: d[k][[0, 2]].contiguous() for k in ("x", "y", "gate", "dh", "dn")}
    r1 = qm.moe_block_norm(one["x"], one["y"], gate=one["gate"], stats=True, **kw)
    b1 = qm.moe_block_norm_backward(one["x"], one["y"], r1.rstd, one["dh"], one["dn"], gate=one["gate"], **kw)
    for got, want in ((r.h, r1.h), (r.n, r1.n), (b.dx, b1.dx), (b.dy, b1.dy), (b.dgate, b1.dgate)):
        assert torch.equal(got[[0, 2]], want) and got[[1, 3]].isnan().all()


@pytest.mark.parametrize("D", [96, 97])
def test_gates_far_out(D):
    # a sigmoid of +-inf and of numbers whose exponent overflows is 1 or 0; NaN stays NaN in its row
    gate = torch.tensor([float("inf"), -float("inf"), 3e38, -3e38, 100.0, -100.0, 0.0, -0.0, float("nan"), 1.0])
    T = gate.numel()
    c = make(T, D, torch.float32)
    d = gpu(c)
    kw = dict(w_post=d["w_post"], gate=gate.cuda(), gate_kind="token", gate_act="sigmoid", w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], eps=1e-5, stats=True, **kw)
    w = {k: ref.f64(v) for k, v in c.items()}
    h, n, mag = ref.norm_forward(w["x"], w["y"], w["w_post"], gate.double(), "token", "sigmoid", 1.0, w["w_pre"], 1e-5)
    fine = ~torch.isnan(gate)
    close(r.h[fine.cuda()], h[fine], mag[fine])
    assert torch.isnan(r.h[~fine.cuda()]).all() and torch.isnan(r.n[~fine.cuda()]).all()
    b = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"], d["dn"], **kw)
    want, m = ref.norm_backward(w["x"][fine], w["y"][fine], w["w_post"], gate.double()[fine], "token", "sigmoid", 1.0, w["w_pre"],
                                1e-5, w["dh"][fine], w["dn"][fine])
    for k in ("dx", "dy", "dgate"):
        close(getattr(b, k)[fine.cuda()], want[k], 3 * m[k], 1e-30)


@pytest.mark.parametrize("T,D", [(1, 32), (3, 512), (5, 544), (17, 3584), (2, 16384)])
@pytest.mark.parametrize("kind", ["fp8", "fp4", "i8"])
def test_codes(T, D, kind):
    # each code is the nearest of the values of its scale to the float64 n, up to the fp32 error of n
    c = make(T, D, kind="channel", seed=2)
    d = gpu(c)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_kind="channel", w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], q_dtype=kind, **kw)
    plain = qm.moe_block_norm(d["x"], d["y"], **kw)
    assert torch.equal(plain.n, r.n) and torch.equal(plain.h, r.h)
    only = qm.moe_block_norm(d["x"], d["y"], q_dtype=kind, want_n=False, **kw)
    assert only.n is None and torch.equal(only.q, r.q) and torch.equal(only.q_scale, r.q_scale)
    w = {k: ref.f64(v) for k, v in c.items()}
    h, n, mag = ref.norm_forward(w["x"], w["y"], w["w_post"], w["gate"], "channel", "none", 1.0, w["w_pre"], 1e-6)
    rh = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
    err = ARITH * (2 * mag * rh + h.abs() * rh) * w["w_pre"].abs()
    if kind == "i8":
        amax = n.abs().amax(1)
        scale = ref.f64(r.q_scale)
        assert ((scale - amax / 127).abs() <= (err.amax(1) + 4 * ref.HALF_F32 * amax) / 127).all()
        v = ref.f64(r.q) * scale[:, None]
        assert (v - n).abs().le(scale[:, None] * (0.5 + 127 * 4 * ref.HALF_F32) + err).all()
        return
    s = r.q_scale.cpu().int() - 127
    b, eb = n.view(T, -1, 32), err.view(T, -1, 32)
    emax, top = (8, 448.0) if kind == "fp8" else (2, 6.0)
    amax, ea = b.abs().amax(2), eb.amax(2)
    lo, hi = (torch.floor(torch.log2(a)) - emax for a in (amax - ea, amax + ea))
    assert ((s >= lo) & (s <= hi)).all()
    unit = torch.exp2(s.double())[..., None]
    if kind == "fp8":
        val = torch.from_numpy(mx.e4m3_value(r.q.cpu().numpy().astype(int) & 127)).view(T, -1, 32)
        sign = torch.where(r.q.cpu() >= 128, -1.0, 1.0).view(T, -1, 32)
        half = torch.maximum(val * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
    else:
        codes = torch.from_numpy(mx.unpack_fp4(r.q.cpu().numpy()).astype(int))
        val = torch.from_numpy(mx.e2m1_value((codes & 7).numpy())).view(T, -1, 32)
        sign = torch.where(codes >= 8, -1.0, 1.0).view(T, -1, 32)
        half = torch.where(val >= 4, 1.0, torch.where(val >= 2, 0.5, 0.25))   # larger side of each code
    off = (sign * val * unit - b).abs()
    saturated = (val == top) & (b.abs() > top * unit - eb)
    assert (off <= half * unit + eb)[~saturated].all()
    assert ((b * sign)[val > 0] >= -eb[val > 0]).all()


@pytest.mark.parametrize("kind", ["fp8", "fp4", "i8"])
def test_codes_are_those_of_the_quantization_of_the_same_values(kind):
    # rows of +-1 have rms 1 and an eps below the last place, so n is +-w_pre exactly: with weights
    # that bf16 holds, the codes must equal those of the call that quantizes bf16 rows
    T, D = 7, 1024
    g = torch.Generator().manual_seed(3)
    x = (torch.randint(0, 2, (T, D), generator=g) * 2 - 1).to(torch.bfloat16).cuda()
    w = (torch.randn(D, generator=g) * torch.exp(2 * torch.randn(D, generator=g))).to(torch.bfloat16)
    r = qm.moe_block_norm(x, w_pre=w.float().cuda(), eps=1e-12, q_dtype=kind)
    assert torch.equal(r.n, x * w.cuda())
    q, s = qm.moe_quant_i8(r.n) if kind == "i8" else qm.moe_quant_act(r.n, kind)
    assert torch.equal(r.q, q) and torch.equal(r.q_scale, s)


def test_no_tokens():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    r = qm.moe_block_norm(x, x, w_post=w, w_pre=w, stats=True)
    assert r.n.shape == (0, 64)
    b = qm.moe_block_norm_backward(x, x, r.rstd, x, x, w_post=w, w_pre=w)
    assert (b.dw_post == 0).all() and (b.dw_pre == 0).all()


@pytest.mark.parametrize("T,D,x_dt", [(7, 11, torch.bfloat16), (600, 515, torch.float32), (3, 5127, torch.bfloat16), (300, 8200, torch.float32)])
def test_gradient_into_a_tensor_of_the_callers(T, D, x_dt):
    d = gpu(make(T, D, x_dt, kind="element", act="sigmoid", seed=7))
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_kind="element", gate_act="sigmoid", w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], stats=True, **kw)
    b = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"], d["dn"], **kw)
    buf = torch.full((T + 2, D), 7.0, dtype=x_dt, device="cuda")
    for dh in (d["dh"], buf[1:-1]):                            # another tensor, and dh itself
        buf[1:-1].copy_(d["dh"])
        o = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, dh, d["dn"], dx=buf[1:-1], **kw)
        assert o.dx.data_ptr() == buf[1:-1].data_ptr()
        assert all(torch.equal(got, want) for got, want in zip(o, b))
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    for bad in (buf, buf[1:-1].t(), torch.empty(T, D, dtype=torch.float16, device="cuda"), torch.empty(T, D, dtype=x_dt)):
        with pytest.raises(ValueError, match="dx"):
            qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"], d["dn"], dx=bad, **kw)
