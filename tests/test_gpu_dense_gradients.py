"""Gradients against differences of the library's own forward pass: a linear layer in microscaled products,
where both are exact, and layer norm with a gradient of the residual stream."""
import math

import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu


def whole(lo, hi, *shape, seed):
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed)).float().cuda()


@pytest.mark.parametrize("T,N,K", [(2, 40, 300), (33, 129, 257), (300, 200, 500), (1000, 520, 640)])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_linear_layer(T, N, K, kind):
    # whole numbers up to 3 are coded without loss whatever their block's largest one, sums of their products (up
    # to 9 times 1000) are exact, and so is the layer's change along any direction: <dY, Y(X + V) - Y(X)> = <dX, V>
    x, w, dy = whole(-2, 2, T, K, seed=1), whole(-2, 2, N, K, seed=2), whole(-3, 3, T, N, seed=3)
    vx, vw = whole(-1, 1, T, K, seed=4), whole(-1, 1, N, K, seed=5)

    def forward(x, w):
        a, b = qm.moe_quant_mx(x, kind), qm.moe_quant_mx(w, "fp4", packed=True)
        return qm.moe_gemm_mx(a.q, a.q_scale, kind, b.q, b.q_scale, N, out_dtype=torch.float32).double()
    d = qm.moe_quant_mx(dy, kind, t_dtype=kind)
    wt = qm.moe_quant_mx(w, t_dtype="fp4", t_packed=True)
    xt = qm.moe_quant_mx(x, t_dtype="fp4", t_packed=True)
    dx = qm.moe_gemm_mx(d.q, d.q_scale, kind, wt.t, wt.t_scale, K, out_dtype=torch.float32).double()
    dw = qm.moe_gemm_mx(d.t, d.t_scale, kind, xt.t, xt.t_scale, K, out_dtype=torch.float32).double()
    y = forward(x, w)
    assert (dy.double() * (forward(x + vx, w) - y)).sum() == (dx * vx.double()).sum() != 0
    assert (dy.double() * (forward(x, w + vw) - y)).sum() == (dw * vw.double()).sum() != 0
    # and entry by entry: a step in one column of X, in one row of W
    e = torch.zeros_like(x)
    e[:, K // 2] = 1
    assert torch.equal((dy.double() * (forward(x + e, w) - y)).sum(1), dx[:, K // 2])
    e = torch.zeros_like(w)
    e[N // 3] = vw[N // 3]
    assert (dy.double() * (forward(x, w + e) - y)).sum() == (dw[N // 3] * vw[N // 3].double()).sum()


@pytest.mark.parametrize("T,D", [(3000, 96), (700, 513), (40, 9000)])
@pytest.mark.parametrize("with_y", [False, True])
def test_layer_norm(T, D, with_y):
    g = torch.Generator().manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x, w, b, dh, dn = 2 * n(T, D), 1 + 0.2 * n(D), 0.3 * n(D), n(T, D), n(T, D).bfloat16()
    y = n(T, D).bfloat16() if with_y else None
    dev = lambda t: None if t is None else t.cuda()   # noqa: E731
    st = qm.moe_layer_norm(dev(x), dev(y), w=dev(w), b=dev(b), stats=True).stats
    d = qm.moe_layer_norm_backward(dev(x), dev(y), st, dev(dh), dev(dn), w=dev(w))
    # along the gradients, each scaled to elements of about 1 (w, b: 1/4)
    v = [t.float().cpu() / float(t.float().square().mean().sqrt()) for t in (d.dx, d.dw, d.db)]
    v = [v[0], v[1] / 4, v[2] / 4]

    def value(f, step):
        return f(*(t + step * u for t, u in zip((x, w, b), v)))

    def library(x, w, b):                                      # sum(h dh) + sum(n dn); h is x where there is no y
        r = qm.moe_layer_norm(x.cuda(), dev(y), w=w.cuda(), b=b.cuda(), want_n=True)
        h = x.cuda() if r.h is None else r.h
        return float((h.double() * dev(dh).double()).sum() + (r.n.double() * dev(dn).double()).sum())

    def definition(x, w, b):
        h, r = ref.layer_norm(x.double().cuda(), None if y is None else y.double().cuda(), w.double().cuda(), b.double().cuda(), 1e-5)
        return float((h * dev(dh).double()).sum() + (r * dev(dn).double()).sum())

    def slope(f, t):                                           # central differences of t and t / 2: off by t^4
        wide, near = (value(f, t) - value(f, -t)) / (2 * t), (value(f, t / 2) - value(f, -t / 2)) / t
        return (4 * near - wide) / 3
    t = 0.1
    gx, gw, gb = (u.double().cpu() for u in (d.dx, d.dw, d.db))
    got = float((gx * v[0].double()).sum() + (gw * v[1].double()).sum() + (gb * v[2].double()).sum())
    # what the difference itself is off by, from the definition in 64 bits
    leaves = [u.double().cuda().requires_grad_(True) for u in (x, w, b)]
    h, r = ref.layer_norm(leaves[0], None if y is None else y.double().cuda(), leaves[1], leaves[2], 1e-5)
    grads = torch.autograd.grad((h, r), leaves, (dev(dh).double(), dev(dn).double()))
    exact = sum(float((a * u.double().cuda()).sum()) for a, u in zip(grads, v))
    off = abs(slope(definition, t) - exact)
    # roundings: of n to bf16, independent, uniform in a half step of 2^-8 |n| (deviation 1 / sqrt(3) of it): six deviations of
    # the sum with the difference's weights 4/3 / t and 1/6 / t, twice each; h, x and the sums of fp32 have 2^-24
    each = float((dn.double().square() * (r.detach().cpu() * ref.HALF_BF16).square()).sum().sqrt()) / math.sqrt(3)
    noise = 6 * each * math.sqrt(2 * (4 / 3 / t) ** 2 + 2 * (1 / 6 / t) ** 2)
    noise += 8 * ref.HALF_F32 / t * float((h.detach().cpu().abs() * dh.double().abs()).sum())
    assert noise + off < 2e-3 * abs(exact)                     # the test can see an error of that size
    assert abs(slope(library, t) - got) <= noise + off + 1e-5 * abs(exact)
