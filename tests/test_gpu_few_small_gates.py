"""The activation of the routed layer of a few tokens from gates and ups of 1 down to 2^-24, each intermediate
value by itself: the second weights select it, so no larger one hides it, and the bound is relative to it."""
import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
E, D, I = 8, 256, 128
BETA, LINEAR_BETA = 4.0, 25.0


def weights(k, seed):
    """(packed weights, float64 values of the gate and up rows [E, 2 I, D]): sums of 256 elements about
    2^(5.6 - 6 - k), and second weights whose row c < I is one in column c."""
    g = torch.Generator().manual_seed(seed)
    w1 = torch.randint(0, 16, (E, 2 * I, D), generator=g, dtype=torch.int32).to(torch.uint8)
    s1 = torch.full((E, 2 * I, D // 32), 127 - 6 - k, dtype=torch.uint8)
    w2 = torch.zeros(E, D, I, dtype=torch.uint8)
    w2[:, torch.arange(I), torch.arange(I)] = 2                # e2m1 code of 1
    s2 = torch.full((E, D, I // 32), 127, dtype=torch.uint8)
    pair = lambda w: ref.pairs(w.flatten(0, 1)).view(E, w.shape[1], -1).contiguous().cuda()   # noqa: E731
    val = ref.mx_values(w1.flatten(0, 1), s1.flatten(0, 1), "fp4").view(E, 2 * I, D)
    return (qm.moe_pack_w1(pair(w1)), s1.cuda(), qm.moe_pack_w2(pair(w2)), s2.cuda()), val


def coded(y, kind):
    return ref.mx_values(*ref.mx_codes(y, kind), kind)


@pytest.mark.parametrize("a", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,K", [(2, 3), (6, 2), (12, 5)])     # one launch for choice and Stage1; two; the rows' sums apart
@pytest.mark.parametrize("k", [0, 4, 8, 12, 16, 20, 24])
def test_small_gates(a, T, K, k):
    w, val = weights(k, 100 * T + k)
    g = torch.Generator().manual_seed(T + K)
    # tokens of +-1: coded without loss, and gate and up sums are exact in any order, also in the matrix
    # instruction's fixed point (products of one size range of 12)
    x = (2 * torch.randint(0, 2, (T, D), generator=g) - 1).bfloat16()
    xa, xs = (x.cuda(), None) if a == "bf16" else qm.moe_quant_act(x.cuda(), a)
    logits = torch.randn(T, E, generator=g).cuda()
    for act in ("situv2", "silu"):
        kw = dict(beta=BETA, linear_beta=LINEAR_BETA) if act == "situv2" else {}
        r = qm.moe_routed_few(logits, xa, xs, a, *w, K, act=act, **kw)
        ids, wk = r.ids.cpu().long(), r.w.cpu().double()
        sums = torch.matmul(val[ids.reshape(-1)], x.double().repeat_interleave(K, 0).unsqueeze(2)).squeeze(2)
        y = ref.activated(sums, act, BETA, LINEAR_BETA)        # [T K, I]
        gate = sums[:, :I]
        dy = 32 * ref.HALF_F32 * (1 + gate.abs()) * y.abs()    # exponentials, quotients, products: a few steps each
        if act == "situv2":
            # each of the two 1 - exp: next to 0 a series, off by x^2 / 6 for x < 2^-7 ln 2, 2^-17.6 of it; beyond, one
            # step of 2^-24 of the exponential beside at least 2^-7.5
            dy = dy + 2 * 2.0 ** -16.5 * y.abs()
        if a == "bf16":
            mid, dy = y, dy + 2.0 ** -16 * y.abs()             # stored in two bf16 parts
        else:
            # the codes, and where y's error reaches a border those on its other side
            mid = coded(y, a)
            dy = torch.maximum((coded(y + dy, a) - mid).abs(), (coded(y - dy, a) - mid).abs())
        wide = wk.reshape(-1, 1)
        want = (mid * wide).view(T, K, I).sum(1)
        err = ((dy + (K + 2) * ref.HALF_F32 * mid.abs()) * wide).view(T, K, I).sum(1)
        got = r.out.cpu().double()
        over = (got[:, :I] - want).abs() - ref.HALF_BF16 * want.abs() - 1.01 * err
        assert (over <= 0).all(), (act, int((over > 0).sum()), float(((got[:, :I] - want).norm() / want.norm())))
        assert (got[:, I:] == 0).all()
