"""The routed layer of a few tokens: choice and weights against float64; the output of bf16 tokens
against float64; that of coded tokens against moe_sort and moe_fused on the same ids and weights (which the
oracle tests hold to float64), up to the roundings that those have besides."""
import numpy as np
import pytest
import torch

import _dense_ref as dref
import _layer_ref as lref
import quantized_moe_expert_sort_amd as qm
from oracle import moe as om
from quantized_moe_expert_sort_amd import inputs as gen

pytestmark = pytest.mark.gpu
SITU = dict(act="situv2", beta=gen.BETA, linear_beta=gen.LINEAR_BETA)
_cache = {}


def weights(E, D, I):
    if (E, D, I) not in _cache:
        _cache.clear()
        g = torch.Generator(device="cuda").manual_seed(E + D + I)
        b = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)   # noqa: E731
        e = lambda lo, *s: torch.randint(lo, lo + 3, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)   # noqa: E731
        w1, w2 = b(E, 2 * I, D // 2), b(E, D, I // 2)
        s1, s2 = e(119, E, 2 * I, D // 32), e(119, E, D, I // 32)
        val = lambda w, s: dref.mx_values(dref.unpairs(w.flatten(0, 1)), s.flatten(0, 1), "fp4").view(E, w.shape[1], -1)   # noqa: E731
        _cache[E, D, I] = (qm.moe_pack_w1(w1), s1, qm.moe_pack_w2(w2), s2), (val(w1, s1), val(w2, s2))
    return _cache[E, D, I]


def float64_output(x, ids, w, values, begin, act):
    """(out [T, D], bound of its error before the last rounding) by the formulas."""
    w1, w2 = values
    E, D, I = w2.shape
    T, K = ids.shape
    out, err = torch.zeros(T, D, dtype=torch.float64, device="cuda"), torch.zeros(T, D, dtype=torch.float64, device="cuda")
    u24 = 2.0 ** -24
    for t in range(T):
        xt = x[t].double()
        for k in range(K):
            e = int(ids[t, k]) - begin if int(ids[t, k]) >= 0 else -1
            if not 0 <= e < E:
                continue
            r, mag = w1[e] @ xt, w1[e].abs() @ xt.abs()
            g, u, (mg, mu) = r[:I], r[I:], (2 * u24 * (D / 32 + 16) * mag).split(I)   # roundings of the sums
            s = torch.sigmoid(g)
            if act == "silu":
                y = g * s * u
                dy = 32 * u24 * (1 + g.abs()) * y.abs()
            else:
                tg, tu = torch.tanh(g / 4), torch.tanh(u / 25)
                y = 100 * tg * s * tu
                dy = 32 * u24 * 100 * s * (tg.abs() + tu.abs() + (1 + g.abs()) * (tg * tu).abs())   # as _layer_ref.gemm_i8
            # slopes: at most 1.25 |u| for g, |g| for u; two bf16 parts: a half step of a half step
            dy = dy + 1.25 * u.abs() * mg + g.abs() * mu + 2.0 ** -16 * y.abs()
            wk = float(w[t, k])
            out[t] += wk * (w2[e] @ y)
            err[t] += abs(wk) * (w2[e].abs() @ (dy + 2 * u24 * (I / 32 + 16 + K) * y.abs()))
    return out, err


def tokens(T, D, a, seed=0):
    g = torch.Generator().manual_seed(seed + 100 * T + D)
    x = torch.randn(T, D, generator=g).bfloat16().cuda()
    return (x, None) if a == "bf16" else qm.moe_quant_act(x, a)


def check(logits, T, D, I, E, K, a, begin=0, local=None, act=SITU, seed=0, **route):
    local = E if local is None else local
    w, values = weights(local, D, I)
    x, xs = tokens(T, D, a, seed)
    r = qm.moe_routed_few(logits, x, xs, a, *w, K, expert_begin=begin, **route, **act)
    bias, valid = route.get("bias"), route.get("valid")
    score = route.get("score", "softmax")
    want = lref.router_choice(logits, K, score, bias, valid)
    assert torch.equal(r.ids.cpu(), want)
    lm = lref.masked_logits(logits)
    ww, _, _, _ = lref.router_outputs(lm, want, score, route.get("renorm", True), route.get("scale", 1.0),
                                      lref.counted(logits, valid), 0.0, 0.0)
    # the weights' exponentials, sums of at most 2048 of them and quotient, as of moe_router: 1e-5 relative
    assert ((lref.f64(r.w) - ww).abs() <= 1e-5 * ww.abs() + 1e-37).all()
    if a == "bf16":
        out, err = float64_output(x, r.ids.cpu(), r.w.cpu(), values, begin, act["act"])
        assert ((r.out.double() - out).abs() <= lref.HALF_BF16 * out.abs() + 1.01 * err).all()
    else:
        lay = qm.moe_sort(r.ids, r.w, begin, local, 16)

        def fused(weight):
            return qm.moe_fused(x, xs, a, *w, weight, lay, local, act["act"], act.get("beta"), act.get("linear_beta")).double()
        # the same codes in between; moe_fused rounds each weighted row, and the sum as it is rounded here
        rows = sum(fused(r.w * (torch.arange(K, device="cuda") == k)).abs() for k in range(K))
        want = fused(r.w)
        assert ((r.out.double() - want).abs() <= lref.HALF_BF16 * (r.out.double().abs() + want.abs() + 1.01 * rows)).all()
    assert torch.isfinite(r.out.float()).all()
    return r


def normal(T, E, dt=torch.float32, seed=0):
    return (1.5 * torch.randn(T, E, generator=torch.Generator().manual_seed(seed + T + E))).to(dt).cuda()


@pytest.mark.parametrize("a", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,E,K,D,I", [(1, 8, 2, 128, 128), (1, 64, 16, 640, 384), (2, 64, 16, 640, 384), (4, 64, 8, 256, 128),
                                       (3, 40, 6, 896, 256), (4, 5, 5, 128, 512), (5, 40, 6, 128, 128), (16, 64, 16, 512, 128),
                                       (16, 64, 2, 512, 128), (16, 300, 32, 128, 128), (1, 300, 32, 128, 128), (13, 33, 1, 256, 384),
                                       (4, 64, 16, 128, 256), (2, 300, 32, 384, 128), (16, 20, 4, 256, 640), (9, 12, 12, 640, 1152)])
def test_shapes_and_types(a, T, E, K, D, I):
    check(normal(T, E), T, D, I, E, K, a)
    check(normal(T, E, torch.bfloat16), T, D, I, E, K, a, act=dict(act="silu"))


@pytest.mark.parametrize("T", [1, 4, 9])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_scores_bias_scale(T, score, renorm):
    bias = (0.05 * torch.randn(100, generator=torch.Generator().manual_seed(5))).cuda()
    for b in (None, bias):
        check(normal(T, 100), T, 128, 128, 100, 7, "bf16", score=score, renorm=renorm, scale=2.5, bias=b)


@pytest.mark.parametrize("E,K", [(1000, 8), (1024, 3), (1025, 8), (2048, 8), (2047, 32)])
@pytest.mark.parametrize("T", [1, 16])
def test_many_experts(E, K, T):
    check(normal(T, E), T, 128, 128, E, K, "bf16")
    bias = (0.01 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()
    check(normal(T, E, torch.bfloat16), T, 128, 128, E, K, "fp8", score="sigmoid", bias=bias)


@pytest.mark.parametrize("T", [3, 12])
def test_masks_and_padding(T):
    l = normal(T, 50)
    l[0] = -float("inf")                                       # nothing left
    l[1, 3:] = -float("inf")                                   # fewer experts than topk
    l[2, 7], l[2, 9] = float("nan"), float("inf")
    valid = torch.ones(T, dtype=torch.bool, device="cuda")
    r = check(l, T, 128, 128, 50, 6, "bf16")
    assert (r.out[0] == 0).all() and (r.ids[0] == -1).all() and (r.w[0] == 0).all()
    valid[T - 1] = False
    r = check(l, T, 128, 128, 50, 6, "fp4", valid=valid)
    assert (r.out[T - 1] == 0).all() and (r.ids[T - 1] == -1).all()
    check(torch.full_like(l, -float("inf")), T, 128, 128, 50, 6, "bf16")
    check(torch.zeros_like(l), T, 128, 128, 50, 6, "bf16")     # ties: the lowest experts
    check(torch.zeros_like(l), T, 128, 128, 50, 6, "bf16", score="sigmoid", bias=torch.zeros(50, device="cuda"))


@pytest.mark.parametrize("T", [2, 4, 10])
@pytest.mark.parametrize("begin,local", [(0, 20), (15, 30), (63, 1), (-4, 10), (60, 40)])
def test_local_experts(T, begin, local):
    check(normal(T, 64), T, 256, 128, 64, 8, "bf16", begin=begin, local=local)


def test_same_expert_for_all():
    l = normal(16, 64)
    l[:, 11] += 40.0
    check(l, 16, 256, 128, 64, 4, "fp8")
    check(l[:4].contiguous(), 4, 256, 128, 64, 4, "fp8")


def test_against_the_oracle():
    E, D, I, K, T = 16, 256, 128, 4, 3
    host = gen.make_weights(3, E, D, I)
    dev = qm.device_weights(*host)
    l = normal(T, E)
    x, _ = tokens(T, D, "bf16")
    r = qm.moe_routed_few(l, x, None, "bf16", *dev, K, **SITU)
    bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    want = om.moe_fused(bits, "bf16", *host, r.ids.cpu().numpy(), r.w.cpu().numpy(), 0, E, "situv2", gen.BETA, gen.LINEAR_BETA)
    assert om.rel_l2(r.out.float().cpu().numpy(), want) < 5e-3


def test_caller_buffers_and_no_tokens():
    w, _ = weights(8, 128, 128)
    x, _ = tokens(2, 128, "bf16")
    out = torch.full((4, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    ws = torch.full((qm.routed_few_ws_bytes(2, 2, 8, 128, 128, 0),), 255, device="cuda", dtype=torch.uint8)
    r = qm.moe_routed_few(normal(2, 8), x, None, "bf16", *w, 2, out=out[:2], ws=ws, **SITU)
    assert r.out.data_ptr() == out.data_ptr() and (out[2:] == 3.0).all()
    assert torch.equal(qm.moe_routed_few(normal(2, 8), x, None, "bf16", *w, 2, **SITU).out, out[:2])
    e = qm.moe_routed_few(normal(2, 8)[:0], x[:0], None, "bf16", *w, 2, **SITU)
    assert e.out.shape == (0, 128)
    with pytest.raises(qm.MoeError, match="WORKSPACE"):
        qm.moe_routed_few(normal(2, 8), x, None, "bf16", *w, 2, ws=ws[:-1], **SITU)


@pytest.mark.parametrize("T", [3, 12])
def test_bad_values_stay_in_their_token(T):
    # every token takes the same experts, so that a bad one shares its tiles with the others
    l = torch.zeros(T, 16, device="cuda")
    w, _ = weights(16, 128, 128)
    x, _ = tokens(T, 128, "bf16")
    clean = qm.moe_routed_few(l, x, None, "bf16", *w, 8, **SITU).out
    for value in (float("nan"), float("inf")):
        bad = x.clone()
        bad[1, 5] = value
        out = qm.moe_routed_few(l, bad, None, "bf16", *w, 8, **SITU).out
        rest = torch.arange(T) != 1
        assert not torch.isfinite(out[1].float()).all() and torch.equal(out[rest], clean[rest])
