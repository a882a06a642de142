"""Gradients through sigmoids far from 0.  The slope is s(g) s(-g): formed as s (1 - s) it loses a digit
with every 2.3 of a positive g and is 0 from 17 on, while the same g with the other sign keeps all.
Against the formulas in float64 with both factors taken as sigmoids, the bounds of the norm's and the
router's tests, and magnitudes that hold the slope too."""
import math

import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
POINTS = (0.5, 3.0, 8.0, 12.0, 15.5, 16.0, 20.0, 30.0, 60.0)


def spread_points(shape, seed):
    """Every point with both signs, in a random order, repeated over the shape."""
    g = torch.Generator().manual_seed(seed)
    n = math.prod(shape)
    p = torch.tensor([s * v for v in POINTS for s in (1.0, -1.0)]).repeat(n // (2 * len(POINTS)) + 1)[:n]
    return p[torch.randperm(n, generator=g)].view(shape)


def within(got, want, mag, arith):
    got = ref.f64(got)
    tol = ref.half_step(got.dtype) * want.abs() + arith * mag
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("x_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["channel", "token", "element"])
@pytest.mark.parametrize("T,D", [(40, 40), (40, 776), (40, 1003), (36, 9000)])
def test_block_norm(kind, T, D, x_dt):
    g = torch.Generator().manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    c = {"x": (3 * n(T, D)).to(x_dt), "y": n(T, D).to(torch.bfloat16), "w_post": 1 + 0.3 * n(D), "w_pre": 1 + 0.3 * n(D),
         "dh": n(T, D).to(x_dt), "dn": n(T, D).to(torch.bfloat16)}
    gate = spread_points({"channel": (D,), "token": (T,), "element": (T, D)}[kind], D)
    gate = gate.to(torch.bfloat16 if kind == "element" else torch.float32)
    d = {k: v.cuda() for k, v in c.items()}
    kw = dict(w_post=d["w_post"], gate=gate.cuda(), gate_kind=kind, gate_act="sigmoid", scale=0.7, w_pre=d["w_pre"])
    r = qm.moe_block_norm(d["x"], d["y"], eps=1e-5, stats=True, **kw)
    b = qm.moe_block_norm_backward(d["x"], d["y"], r.rstd, d["dh"], d["dn"], **kw)
    # the gradient for s = sigmoid(gate) taken as a raw gate, then the slope
    w = {k: ref.f64(v) for k, v in c.items()}
    s, slope = torch.sigmoid(gate.double()), torch.sigmoid(gate.double()) * torch.sigmoid(-gate.double())
    want, m = ref.norm_backward(w["x"], w["y"], w["w_post"], s, kind, "none", 0.7, w["w_pre"], 1e-5, w["dh"], w["dn"])
    within(b.dgate, want["dgate"] * slope, 3 * m["dgate"] * slope, 64 * ref.HALF_F32 + ref.half_step(b.dgate.dtype))
    for k in ("dx", "dy", "dw_post", "dw_pre"):
        got = getattr(b, k)
        within(got, want[k], 3 * m[k], 64 * ref.HALF_F32 + ref.half_step(got.dtype))


@pytest.mark.parametrize("E,K", [(24, 4), (257, 8), (896, 16), (1100, 8)])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_sigmoid_scores(E, K, renorm):
    # rows from wholly saturated to mixed; REL as in the router's tests
    T, rel = 24, 128 * ref.HALF_F32
    logits = spread_points((T, E), E)
    logits[:4] = logits[:4].abs().clamp(min=8.0) + 0.001 * torch.arange(E)
    g = torch.Generator().manual_seed(E)
    dw = torch.randn(T, K, generator=g)
    kw = dict(score="sigmoid", renorm=renorm, scale=1.5)
    r = qm.moe_router(logits.cuda(), K, balance=(0.4, 0.0), **kw)
    ids = r.ids.cpu().long()
    l = logits.double()
    s, rest = torch.sigmoid(l), torch.sigmoid(-l)
    # the weights' part
    sk, gk = s.gather(1, ids), dw.double()
    v = sk / sk.sum(1, keepdim=True) if renorm else sk
    mean = (v * gk).sum(1, keepdim=True) if renorm else torch.zeros(T, 1, dtype=torch.float64)
    size = (v * gk.abs()).sum(1, keepdim=True) if renorm else torch.zeros(T, 1, dtype=torch.float64)
    own = torch.zeros(T, E, dtype=torch.float64).scatter(1, ids, 1.5 * v * (gk - mean)) * rest
    own_m = torch.zeros(T, E, dtype=torch.float64).scatter(1, ids, 1.5 * v * (gk.abs() + size)) * rest
    got = qm.moe_router_backward(logits.cuda(), r._replace(balance=None), dw.cuda(), **kw)
    bad = (ref.f64(got) - own).abs() > rel * own_m + ref.HALF_F32 * own.abs()
    assert not bad.any(), (int(bad.sum()), l[bad][:8].tolist())
    # and the balance loss's, with a gradient of 2 for it
    a = 2.0 * 0.4 * torch.bincount(ids.flatten(), minlength=E) * E / (K * T * T)
    p = s / s.sum(1, keepdim=True)
    am = (a * p).sum(1, keepdim=True)
    want, m = own + p * rest * (a - am), own_m + p * rest * (a + am)
    got = qm.moe_router_backward(logits.cuda(), r, dw.cuda(), d_loss=torch.tensor([2.0, 0.0]).cuda(), **kw)
    bad = (ref.f64(got) - want).abs() > 2 * rel * m + ref.HALF_F32 * want.abs()
    assert not bad.any(), (int(bad.sum()), l[bad][:8].tolist())
