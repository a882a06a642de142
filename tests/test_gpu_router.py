"""moe_router and its backward pass against float64: the chosen experts have to be equal, weights,
statistics and gradients within bounds counted from the fp32 roundings."""
import math

import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
# exp2 of an fp32 product: an exponent of up to 64 rounds by 64 * 2^-24, the rest of a probability
# (exp2 itself, sums of up to 32 + 6 terms a lane and wave, the quotient) by 64 roundings more
REL = 128 * ref.HALF_F32


def make(T, E, dt=torch.float32, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + E)
    return (spread * torch.randn(T, E, generator=g)).to(dt), g


def close(got, want, tol, what):
    bad = (ref.f64(got) - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((ref.f64(got) - want).abs() / tol.clamp(min=1e-300)).max()))


def check(logits, K, score="softmax", renorm=True, scale=1.0, bias=None, valid=None, coef=0.3, z_coef=0.02, train=True,
          seed=0, d_loss=(0.7, 1.3)):
    T, E = logits.shape
    cuda = lambda t: None if t is None else t.cuda()   # noqa: E731
    d_logits, b, v = logits.cuda(), cuda(bias), cuda(valid)
    kw = dict(score=score, renorm=renorm, scale=scale, valid=v)
    plain = qm.moe_router(d_logits, K, bias=b, **kw)
    ids = ref.router_choice(logits, K, score, bias, valid)
    assert torch.equal(plain.ids.cpu(), ids)
    assert plain.balance is None
    l = ref.masked_logits(logits).requires_grad_(True)
    ok = ref.counted(logits, valid)
    w, counts, mean, loss = ref.router_outputs(l, ids, score, renorm, scale, ok, coef, z_coef)
    close(plain.w, w.detach(), REL * w.detach().abs() + 1e-36, "w")
    if not train:
        return plain
    r = qm.moe_router(d_logits, K, bias=b, balance=(coef, z_coef), **kw)
    assert torch.equal(r.ids, plain.ids) and torch.equal(r.w, plain.w)
    assert torch.equal(r.balance.counts.cpu().long(), counts)
    assert int(r.balance.num_valid) == int(ok.sum())
    # up to 64 rows of a wave and 16 + 16 partial sums are added behind each other
    close(r.balance.mean_prob, mean.detach(), 2 * REL * mean.detach() + 1e-36, "mean_prob")
    close(r.balance.loss, loss.detach(), 4 * REL * loss.detach().abs() + 1e-36, "loss")
    g = torch.Generator().manual_seed(seed + 11)
    dw = torch.randn(T, K, generator=g)
    dl = torch.tensor(d_loss)
    got = qm.moe_router_backward(d_logits, r, dw.cuda(), d_loss=dl.cuda(), **kw)
    total = (w * dw.double()).sum() + (loss * dl.double()).sum()
    want, = torch.autograd.grad(total, l)
    want = torch.nan_to_num(want, nan=0.0)                     # masked entries: no gradient
    # the magnitudes of a gradient's terms: its own weight's, the row's mean, the two losses'
    rows = torch.where(ok[:, None], l.detach(), torch.zeros_like(l))
    soft = torch.softmax(rows, 1)
    on = ids >= 0
    at = ids.clamp(min=0).long()
    wm = w.detach().abs() * (dw.double().abs() + (dw.double() * w.detach()).abs().sum(1, keepdim=True) / max(abs(scale), 1e-9))
    mag = torch.zeros_like(rows).scatter_add(1, at, torch.where(on, wm, 0.0))
    if score == "softmax" and not renorm:
        mag = mag + soft * wm.sum(1, keepdim=True)
    n = max(int(ok.sum()), 1)
    a = d_loss[0] * coef * counts * E / (K * n * n)
    share = torch.softmax(rows if score == "softmax" else torch.nn.functional.logsigmoid(rows), 1)
    mag = mag + share * (a + (a * share).sum(1, keepdim=True))
    mag = mag + soft * abs(d_loss[1] * z_coef) * 2 * torch.logsumexp(rows, 1, keepdim=True).abs() / n
    mag = mag * ok[:, None]
    close(got, want, 4 * REL * mag + ref.half_step(got.dtype) * want.abs() + 1e-36, "d_logits")
    assert (ref.f64(got)[~ok] == 0).all()
    return r


@pytest.mark.parametrize("E,K", [(1, 1), (2, 1), (3, 3), (8, 2), (60, 6), (64, 32), (65, 8), (112, 16), (128, 32), (256, 8),
                                 (257, 4), (264, 32), (512, 8), (896, 16), (1000, 10), (1023, 5), (1024, 32), (1032, 2),
                                 (2047, 16), (2048, 32)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_sizes(E, K, dt):
    logits, g = make(37, E, dt)
    check(logits, K)
    check(logits, K, "sigmoid", bias=0.1 * torch.randn(E, generator=g), scale=2.5)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 64, 255, 4097, 9000])
def test_token_counts(T):
    logits, g = make(T, 96)
    check(logits, 4, valid=torch.rand(T, generator=g) < 0.7)
    check(logits, 4, "sigmoid", renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("E", [100, 896])
def test_combinations(score, renorm, with_bias, E):
    logits, g = make(130, E)
    bias = 0.02 * torch.randn(E, generator=g) if with_bias else None
    check(logits, 7, score, renorm, 1.7, bias, torch.rand(130, generator=g) < 0.9)
    check(logits.bfloat16(), 7, score, renorm, 1.0, bias)


@pytest.mark.parametrize("E", [48, 112, 200, 896, 1500])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_keys_go_to_the_lowest_expert(E, with_bias, score):
    # all equal (more than 64 keys at the border: the slow path), few distinct values, and two runs
    g = torch.Generator().manual_seed(E)
    bias = torch.zeros(E) if with_bias else None
    few = torch.randint(0, 4, (9, E), generator=g).float()
    runs = torch.where(torch.arange(E) % 2 == 0, 1.0, 0.0).repeat(3, 1)
    zeros = torch.where(torch.rand(3, E, generator=g) < 0.5, -0.0, 0.0)
    for logits in (torch.zeros(2, E), few, few.bfloat16(), runs, zeros, torch.full((2, E), -3e38)):
        check(logits, min(E, 16), score, bias=bias, z_coef=0.0 if logits.min() < -1e30 else 0.02)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(100, 32), (130, 31), (512, 32), (800, 28), (1023, 32), (1024, 31), (1536, 32), (2048, 32)])
def test_rows_with_many_candidates(E, K, dt):
    # with K near half the lanes the lanes' maxima bound the choice so loosely that more than 64 experts
    # pass; among 300 rows some do at each of these sizes
    logits, g = make(300, E, dt)
    check(logits, K, train=False)
    check(logits, K, "sigmoid", bias=0.1 * torch.randn(E, generator=g), train=False)
    check(logits, K, "softmax", bias=0.01 * torch.randn(E, generator=g), train=False)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [96, 200, 500, 896, 1021, 2048])
def test_rows_of_ties(E, dt):
    g = torch.Generator().manual_seed(E)
    flat = torch.zeros(8, E)
    flat[1] = -3.5
    flat[2] = 3e38                                             # all at the top
    flat[3, ::2] = -0.0                                        # equal to 0
    flat[4] = torch.randint(0, 2, (E,), generator=g).float()   # two values
    flat[5] = torch.randint(0, 2, (E,), generator=g).float() - 1
    flat[6] = 1.0
    flat[6, torch.randperm(E, generator=g)[:7]] = 2.0          # a few above the ties
    flat[7, torch.randperm(E, generator=g)[:E // 2]] = float("-inf")
    flat = flat.to(dt)
    levels = torch.randint(0, 3, (E,), generator=g).float() / 4
    masked = levels.clone()
    masked[::3] = float("nan")
    masked[1::5] = float("-inf")
    for K in (1, 8, 32):
        check(flat, K, train=False)
        for bias in (torch.zeros(E), levels, masked):
            check(flat, K, "sigmoid", bias=bias, train=False)
            check(flat, K, "softmax", bias=bias, train=False)


def test_keys_that_32_bits_cannot_order():
    # pairs of experts whose keys differ by 1e-9: fp32 rounds them to the same value or swaps them
    E, T = 64, 200
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(T, E, generator=g)
    for score in ("sigmoid", "softmax"):
        s = torch.sigmoid(logits.double()) if score == "sigmoid" else torch.softmax(logits.double(), 1)
        bias = (1.0 - s[0]).float()                            # row 0: every key within 2^-24 of 1
        check(logits, 8, score, bias=bias, train=False)
        check(logits[:1].repeat(40, 1), 8, score, bias=bias, train=False)
        big, gb = make(64, 896, torch.bfloat16, 5)
        check(big, 16, score, bias=torch.zeros(896), train=False)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [96, 640])
def test_masked_experts(dt, score, E):
    T, K = 12, 8
    logits, g = make(T, E, dt, 3)
    low = torch.finfo(dt).min
    logits[0] = -math.inf                                      # nothing left
    logits[1] = -math.inf
    logits[1, 5] = 0.5                                         # one expert left
    logits[2, 3:] = -math.inf                                  # fewer than K
    logits[3, : E - K] = -math.inf                             # exactly K
    logits[4, ::3] = math.nan
    logits[5] = math.nan
    logits[6, :] = -math.inf
    logits[6, E - 1] = -100.0
    valid = torch.ones(T, dtype=torch.bool)
    valid[7] = False
    check(logits, K, score, valid=valid)
    check(logits, K, score, renorm=False, valid=valid.to(torch.uint8))
    bias = 0.1 * torch.randn(E, generator=g)
    bias[:4] = -math.inf
    bias[4] = math.nan
    check(logits, K, score, bias=bias, valid=valid)
    # masks of the type's lowest value stay selectable, after everything else
    logits, _ = make(T, E, dt, 4)
    logits[0] = low
    logits[1, 2:] = low
    check(logits, K, score, z_coef=0.0)
    logits[2, 7], logits[2, 9], logits[3, 1] = math.inf, math.inf, math.inf
    check(logits, K, score, z_coef=0.0)
    bias = torch.zeros(E)
    bias[[2, 9]] = math.inf
    bias[11] = -torch.finfo(torch.float32).max
    check(logits, K, score, bias=bias, z_coef=0.0, train=False)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_infinity_comes_before_the_largest_finite_logit(dt):
    # +inf counts as fp32's largest value, which no bf16 holds: above bf16's largest, level with fp32's
    logits, _ = make(3, 300, dt)
    logits[0, 10], logits[0, 200] = torch.finfo(dt).max, math.inf
    logits[1, 10], logits[1, 200], logits[1, 201] = math.inf, torch.finfo(dt).max, math.inf
    logits[2, :] = torch.finfo(dt).max
    logits[2, 299] = math.inf
    check(logits, 4, z_coef=0.0)
    check(logits, 4, "sigmoid", z_coef=0.0)


def test_no_counted_token():
    logits, _ = make(5, 40)
    r = check(logits, 3, valid=torch.zeros(5, dtype=torch.bool))
    assert (r.ids == -1).all() and (r.balance.loss == 0).all() and (r.balance.counts == 0).all()
    empty = torch.empty((0, 40), device="cuda")
    r = qm.moe_router(empty, 3, balance=(1.0, 1.0))
    assert r.ids.shape == (0, 3) and (r.balance.mean_prob == 0).all() and int(r.balance.num_valid) == 0
    assert qm.moe_router_backward(empty, r).shape == (0, 40)


def test_pointers_that_no_wide_load_may_read():
    logits, _ = make(9, 512, torch.bfloat16)
    moved = torch.cat((logits.new_zeros(1), logits.flatten())).cuda()[1:].view(9, 512)
    assert torch.equal(qm.moe_router(moved, 8).ids.cpu(), ref.router_choice(logits, 8, "softmax"))
    r = qm.moe_router(logits.cuda(), 8, balance=(1.0, 0.1))
    dw = torch.randn(9, 8, device="cuda")
    a, b = qm.moe_router_backward(logits.cuda(), r, dw), qm.moe_router_backward(moved, r, dw)
    assert torch.allclose(a.float(), b.float(), rtol=2 * ref.HALF_BF16, atol=1e-9)


def test_backward_with_ids_of_the_callers_own():
    # an expert named twice gets both parts; ids outside the range none
    E = 50
    logits, _ = make(2, E)
    ids = torch.tensor([[3, 3, 7, -1], [49, 50, -7, 2]], dtype=torch.int32)
    dw = torch.randn(2, 4, generator=torch.Generator().manual_seed(1))
    r = qm.Routing(ids.cuda(), None, None)
    got = qm.moe_router_backward(logits.cuda(), r, dw.cuda(), renorm=False)
    l = logits.double().requires_grad_(True)
    on = (ids >= 0) & (ids < E)
    p = torch.softmax(l, 1).gather(1, torch.where(on, ids, 0).long())
    want, = torch.autograd.grad((p * torch.where(on, dw.double(), 0.0)).sum(), l)
    assert (ref.f64(got) - want).abs().max() < REL


def test_gradients_against_differences():
    T, E, K = 6, 40, 5
    logits, g = make(T, E, seed=2, spread=1.0)
    dw = torch.randn(T, K, generator=g, dtype=torch.float64)
    v = torch.randn(T, E, generator=g, dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            kw = dict(score=score, renorm=renorm, scale=1.5)
            r = qm.moe_router(logits.cuda(), K, balance=(0.5, 0.1), **kw)
            got = qm.moe_router_backward(logits.cuda(), r, dw.float().cuda(), **kw)
            ids = r.ids.cpu()
            ok = torch.ones(T, dtype=torch.bool)

            def value(s):
                w, _, _, loss = ref.router_outputs(logits.double() + s * v, ids, score, renorm, 1.5, ok, 0.5, 0.1)
                return float((w * dw.float().double()).sum() + loss.sum())
            want = (value(1e-4) - value(-1e-4)) / 2e-4
            assert abs(float((ref.f64(got) * v).sum()) - want) < 1e-6 + 8 * REL * float((ref.f64(got) * v).abs().sum())


def test_parts_of_the_gradient_and_repeatability():
    logits, _ = make(300, 896)
    x = logits.cuda()
    dw = torch.randn(300, 16, device="cuda")
    r = qm.moe_router(x, 16, balance=(0.4, 0.1))
    both = qm.moe_router_backward(x, r, dw)
    zero = qm.moe_router_backward(x, r, dw, d_loss=torch.zeros(2, device="cuda"))
    only = qm.moe_router_backward(x, r)
    alone = qm.moe_router_backward(x, r._replace(balance=None), dw)
    assert torch.allclose(zero, alone, rtol=1e-5, atol=1e-9)
    assert torch.allclose(both, alone + only, rtol=1e-4, atol=1e-8)
    for _ in range(3):
        s = qm.moe_router(x, 16, balance=(0.4, 0.1))
        assert all(torch.equal(a, b) for a, b in zip((s.ids, s.w, *s.balance[:4]), (r.ids, r.w, *r.balance[:4])))
        assert torch.equal(qm.moe_router_backward(x, r, dw), both)
