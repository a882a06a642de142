"""Layer norm and its backward pass against float64, at every kind of width, type and option."""
import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

CASES = [  # T, D, type, y, w, b
    (1, 3584, "bf16", True, True, True), (1, 1, "f32", False, True, True), (5, 7, "bf16", True, True, False),
    (3, 8, "f32", True, False, False), (70, 64, "f32", False, True, True), (33, 513, "bf16", True, True, True),
    (300, 1790, "bf16", False, True, True), (257, 3584, "f32", True, True, True), (19, 8192, "bf16", True, True, True),
    (6, 8200, "f32", True, True, True), (4, 12001, "bf16", True, True, True), (3, 16384, "f32", False, True, True),
    (2, 16383, "bf16", True, True, True), (2000, 100, "bf16", True, True, True), (1100, 520, "f32", True, True, False),
]


def make(T, D, dt, y, w, b, offset=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + D)
    n = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x = (2 * n(T, D) * torch.exp(0.5 * n(T, 1)) + offset * n(T, 1)).to(TYPES[dt])
    return dict(x=x, y=n(T, D).bfloat16() if y else None, w=1 + 0.2 * n(D) if w else None, b=0.3 * n(D) if b else None,
                dh=n(T, D).to(TYPES[dt]), dn=n(T, D).bfloat16())


def dev(s):
    return {k: None if v is None else v.cuda() for k, v in s.items()}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check_forward(s, r):
    x, y, w, b = (f64(s[k]) for k in ("x", "y", "w", "b"))
    h, n = ref.layer_norm(x, y, w, b, EPS)
    m, rs, z, ez = ref.layer_norm_parts(h, EPS)
    half = ref.half_step(s["x"].dtype)
    if y is not None:
        assert ((f64(r.h) - h).abs() <= half * h.abs() * (1 + 2 * half) + ref.HALF_F32 * h.abs()).all()
    zw = z if w is None else z * w
    err = (ez if w is None else ez * w.abs()) + 2 * ref.HALF_F32 * (zw.abs() + (0 if b is None else b.abs()))
    assert ((f64(r.n) - n).abs() <= ref.HALF_BF16 * n.abs() + 1.01 * err).all()
    dm = 4 * (h.abs().amax(1) + m[:, 0].abs()) + 32 / rs[:, 0]
    assert ((f64(r.stats[0]) - m[:, 0]).abs() <= ref.HALF_F32 * dm).all()
    per_row = ((h.abs() + m.abs()) * rs).amax(1)
    assert ((f64(r.stats[1]) / rs[:, 0] - 1).abs() <= ref.HALF_F32 * (24 + 4 * per_row)).all()


def check_backward(s, d, has_dh=True):
    x, y, w, dh, dn = (f64(s[k]) for k in ("x", "y", "w", "dh", "dn"))
    if not has_dh:
        dh = torch.zeros_like(x)
    h = x if y is None else x + y
    m, r, z, ez = ref.layer_norm_parts(h, EPS)
    u = dn if w is None else dn * w
    mu, mz = u.mean(1, keepdim=True), (u * z).mean(1, keepdim=True)
    e = dh + r * (u - mu - z * mz)
    # sums over a row of up to 32 roundings, a product or two more; z's own error where it enters
    au, az = u.abs().mean(1, keepdim=True), (u * z).abs().mean(1, keepdim=True)
    per_row = ((h.abs() + m.abs()) * r).amax(1, keepdim=True)
    err = ref.HALF_F32 * (2 * dh.abs() + r * (8 * u.abs() + 36 * au + 36 * z.abs() * az))
    err = err + r * (ez * az + z.abs() * (u.abs() * ez).mean(1, keepdim=True))
    err = err + ref.HALF_F32 * (24 + 4 * per_row) * (e - dh).abs()
    half = ref.half_step(s["x"].dtype)
    assert ((f64(d.dx) - e).abs() <= half * e.abs() + 1.01 * err).all()
    if y is not None:
        assert ((f64(d.dy) - e).abs() <= ref.HALF_BF16 * e.abs() + 1.01 * err).all()
    # at most 128 rows in a register, 16 in a workgroup, 256 partial sums in 16 + 16 steps
    adds = 192 * ref.HALF_F32
    if w is not None:
        err = adds * (dn * z).abs().sum(0) + (dn.abs() * ez).sum(0)
        assert ((f64(d.dw) - (dn * z).sum(0)).abs() <= 1.01 * err).all()
    assert ((f64(d.db) - dn.sum(0)).abs() <= adds * dn.abs().sum(0)).all()


@pytest.mark.parametrize("T,D,dt,y,w,b", CASES)
def test_against_float64(T, D, dt, y, w, b):
    s = make(T, D, dt, y, w, b)
    c = dev(s)
    r = qm.moe_layer_norm(c["x"], c["y"], w=c["w"], b=c["b"], eps=EPS, stats=True)
    check_forward(s, r)
    d = qm.moe_layer_norm_backward(c["x"], c["y"], r.stats, c["dh"], c["dn"], w=c["w"])
    check_backward(s, d)
    assert (d.dw is None) == (not w) and (d.dy is None) == (not y)
    if y:
        again = qm.moe_layer_norm(c["x"], c["y"], w=c["w"], b=c["b"], eps=EPS, h=c["x"])   # in place
        assert torch.equal(again.h, r.h) and torch.equal(again.n, r.n) and again.h.data_ptr() == c["x"].data_ptr()


def test_no_stream_gradient_and_in_place():
    s = make(40, 777, "f32", True, True, True)
    c = dev(s)
    st = qm.moe_layer_norm(c["x"], c["y"], w=c["w"], b=c["b"], eps=EPS, stats=True).stats
    d = qm.moe_layer_norm_backward(c["x"], c["y"], st, None, c["dn"], w=c["w"])
    check_backward(s, d, has_dh=False)
    full = qm.moe_layer_norm_backward(c["x"], c["y"], st, c["dh"], c["dn"], w=c["w"])
    into = qm.moe_layer_norm_backward(c["x"], c["y"], st, c["dh"], c["dn"], w=c["w"], bias=False, dx=c["dh"])
    assert into.db is None and into.dx.data_ptr() == c["dh"].data_ptr() and torch.equal(into.dx, full.dx)


def test_gradient_against_differences():
    # a directional difference of the library's own forward pass: sum(n dn) + sum(h dh) along a random direction
    s = make(6, 96, "f32", False, True, True)
    c = dev(s)
    st = qm.moe_layer_norm(c["x"], w=c["w"], b=c["b"], eps=EPS, stats=True).stats
    d = qm.moe_layer_norm_backward(c["x"], None, st, None, c["dn"], w=c["w"])
    dirs = {k: torch.randn(c[k].shape, generator=torch.Generator().manual_seed(i)).cuda() for i, k in enumerate("xwb")}

    def value(step):
        f = {k: f64(c[k]) + step * f64(dirs[k]) for k in "xwb"}
        return float((ref.layer_norm(f["x"], None, f["w"], f["b"], EPS)[1] * f64(c["dn"])).sum())
    t = 1e-4                                                   # central: off by t^2 of the third derivative
    slope = (value(t) - value(-t)) / (2 * t)
    got = float((f64(d.dx) * f64(dirs["x"])).sum() + (f64(d.dw) * f64(dirs["w"])).sum() + (f64(d.db) * f64(dirs["b"])).sum())
    scale = float((f64(d.dx) * f64(dirs["x"])).abs().sum() + (f64(d.dw) * f64(dirs["w"])).abs().sum())
    assert abs(slope - got) <= 1e-5 * scale


def test_large_mean():
    # deviations of 1 beside a mean of 10000: fp32 holds the inputs' deviations to 5e-4 of a deviation; the
    # mean's own rounding must not show in n
    s = make(9, 2000, "f32", False, True, True, offset=0.0)
    s["x"] = (s["x"] / s["x"].std(1, keepdim=True) + 10000.0)
    c = dev(s)
    r = qm.moe_layer_norm(c["x"], w=c["w"], b=c["b"], eps=EPS, stats=True)
    z = (f64(r.n) - f64(s["b"])) / f64(s["w"])
    want = ref.layer_norm(f64(s["x"]), None, None, None, EPS)[1]
    assert float((z - want).mean(1).abs().max()) < 2e-4        # 2000 roundings of n average out
    check_forward(s, r)


def test_constant_rows_and_bad_rows():
    x = torch.randn(6, 136, generator=torch.Generator().manual_seed(1))
    x[1] = 3.25                                                # no deviation: n is the bias
    x[3, 5], x[4, 100] = float("inf"), float("nan")
    w, b = torch.rand(136) + 0.5, torch.randn(136)
    r = qm.moe_layer_norm(x.cuda(), w=w.cuda(), b=b.cuda(), eps=EPS)
    n = r.n.cpu()
    assert torch.equal(n[1], b.bfloat16())
    assert n[3].isnan().all() and n[4].isnan().all() and not n[[0, 1, 2, 5]].isnan().any()


@pytest.mark.parametrize("kind", ["fp8", "fp4", "i8"])
def test_codes(kind):
    s = make(37, 896, "bf16", True, True, True)
    c = dev(s)
    r = qm.moe_layer_norm(c["x"], c["y"], w=c["w"], b=c["b"], eps=EPS, q_dtype=kind, stats=True)
    check_forward(s, r)
    only = qm.moe_layer_norm(c["x"], c["y"], w=c["w"], b=c["b"], eps=EPS, q_dtype=kind, want_n=False)
    assert only.n is None and torch.equal(only.q, r.q) and torch.equal(only.q_scale, r.q_scale)
    n = ref.layer_norm(*(f64(s[k]) for k in ("x", "y", "w", "b")), EPS)[1]
    if kind == "i8":
        amax = n.abs().amax(1, keepdim=True)
        assert ((f64(r.q_scale)[:, None] * 127 / amax - 1).abs() < 1e-5).all()
        # half a code, and what fp32 moves a value by
        assert ((f64(r.q) * amax / 127 - n).abs() <= amax / 127 * (0.5 + 1e-3)).all()
    else:
        codes = ref.unpairs(r.q.cpu()) if kind == "fp4" else r.q.cpu()
        v = ref.mx_values(codes, r.q_scale.cpu(), kind)
        amax = n.view(37, -1, 32).abs().amax(2).repeat_interleave(32, 1)
        # elements: half a step of at most amax / 4 (fp4; saturating from 6 on 8: amax / 4) or amax / 16 (fp8; 448 of 512)
        assert ((v - n).abs() <= amax * (0.25 if kind == "fp4" else 0.125) * (1 + 1e-4)).all()
        want, ws = ref.mx_codes(n, kind)
        assert (r.q_scale.cpu() != ws).float().mean() < 1e-3 and (codes != want).float().mean() < 1e-3


def test_padded_rows_stay():
    # the rows behind a batch's last one are not written
    x = torch.randn(8, 200, device="cuda")
    w = torch.ones(200, device="cuda")
    h = torch.full((8, 200), 7.0, device="cuda")
    y = torch.randn(5, 200, device="cuda").bfloat16()
    qm.moe_layer_norm(x[:5], y, w=w, h=h[:5])
    assert (h[5:] == 7.0).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    r = qm.moe_layer_norm(x, w=w, stats=True)
    assert r.n.shape == (0, 64)
    d = qm.moe_layer_norm_backward(x, None, r.stats, None, r.n, w=w)
    assert (d.dw == 0).all() and (d.db == 0).all()
