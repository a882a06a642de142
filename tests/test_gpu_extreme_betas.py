"""SiTUv2 with every beta and linear_beta that the calls take: large ones, whose product leaves fp32's range and
which make it SiLU, and small ones, whose inverse does, in the products and the routed layer of a few tokens."""
import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
MOST = float(torch.finfo(torch.float32).max)
# the last two: outputs below fp32's smallest number are 0
BETAS = [(4.0, 25.0), (1e6, 1e5), (1e8, 1e8), (1e19, 1e19), (1e20, 1e20), (1e30, 1e30), (MOST, MOST), (MOST, 1.0), (1.0, 1e35), (1e30, 1e-30),
         (1e-37, 25.0), (1e-39, 25.0), (25.0, 1e-42), (1e-39, MOST), (1e-30, 1e-30), (1e-45, 1e-45)]


def close(got, sums, beta, lb, half, more=0.0):
    g, u = sums.chunk(2, 1)
    beta, lb = (float(torch.tensor(v, dtype=torch.float32)) for v in (beta, lb))   # as the call gets them
    want = ref.activated(sums, "situv2", beta, lb)
    # exponentials, quotients and products a few steps each; each 1 - exp to 2^-16.5 of it (a series next to 0,
    # beyond it one step of 2^-24 beside 2^-7.5); steps of numbers below 2^-126 are 2^-149 and may count as 0
    err = (32 * ref.HALF_F32 * (1 + g.abs()) + 2 * 2.0 ** -16.5 + more) * want.abs() + 2.0 ** -126
    over = (got.double() - want).abs() - half * want.abs() - 1.01 * err
    assert (over <= 0).all(), (int((over > 0).sum()), got.flatten()[:4], want.flatten()[:4])


def codes(*shape, seed):
    return torch.randint(0, 16, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int32).to(torch.uint8)


@pytest.mark.parametrize("beta,lb", BETAS)
@pytest.mark.parametrize("T", [1, 100])                        # streamed weights, tiles
@pytest.mark.parametrize("scale", [121, 101])                  # sums of about 1 and of 2^-20
def test_gemm_mx(beta, lb, T, scale):
    a, w = codes(T, 256, seed=T), codes(96, 256, seed=7)
    a[:, 128:] = 0                                             # a gate and an up of 0 too
    w[5], w[60] = 0, 0
    sa, sw = torch.full((T, 8), 127 - 2, dtype=torch.uint8), torch.full((96, 8), scale, dtype=torch.uint8)
    sums = ref.mx_values(a, sa, "fp4") @ ref.mx_values(w, sw, "fp4").t()
    p, ps = qm.moe_pack_mx(ref.pairs(w).cuda(), sw.cuda())
    for dt in (torch.float32, torch.bfloat16):
        out = qm.moe_gemm_mx(ref.pairs(a).cuda(), sa.cuda(), "fp4", p, ps, 96, act="situv2", beta=beta, linear_beta=lb, out_dtype=dt)
        close(out.cpu(), sums, beta, lb, ref.half_step(dt))


@pytest.mark.parametrize("beta,lb", BETAS)
@pytest.mark.parametrize("T", [1, 100])
def test_gemm_i8(beta, lb, T):
    a, w = codes(T, 256, seed=T).to(torch.int8) - 8, codes(96, 256, seed=7).to(torch.int8) - 8
    sa, sw = torch.full((T,), 2.0 ** -8), torch.full((96,), 0.5)
    sums = (a.double() @ w.double().t()) * 2.0 ** -9
    out = qm.moe_gemm_i8(a.cuda(), sa.cuda(), qm.moe_pack_i8(w.cuda()), sw.cuda(), act="situv2", beta=beta, linear_beta=lb)
    close(out.cpu(), sums, beta, lb, ref.HALF_BF16)


@pytest.mark.parametrize("beta,lb", BETAS)
@pytest.mark.parametrize("T", [2, 9])                          # the choice in Stage1's launch, before it
def test_routed_few(beta, lb, T):
    # one expert with weight 1 whose second weights select one value each
    E, D, I = 2, 128, 128
    w1 = codes(2 * I, D, seed=3)
    w1[5], w1[I + 9] = 0, 0
    s1 = torch.full((E, 2 * I, D // 32), 127 - 6, dtype=torch.uint8)
    w2 = torch.zeros(D, I, dtype=torch.uint8)
    w2[torch.arange(I), torch.arange(I)] = 2                   # e2m1 code of 1
    pair = lambda w: ref.pairs(w).expand(E, -1, -1).contiguous().cuda()   # noqa: E731
    x = (2 * codes(T, D, seed=T).remainder(2).float() - 1).bfloat16()
    sums = x.double() @ ref.mx_values(w1, s1[0], "fp4").t()
    logits = torch.zeros(T, E, device="cuda")
    r = qm.moe_routed_few(logits, x.cuda(), None, "bf16", qm.moe_pack_w1(pair(w1)), s1.cuda(), qm.moe_pack_w2(pair(w2)),
                          torch.full((E, D, I // 32), 127, dtype=torch.uint8, device="cuda"), 1, act="situv2", beta=beta, linear_beta=lb)
    assert (r.w == 1).all()
    close(r.out.cpu(), sums, beta, lb, ref.HALF_BF16, more=2.0 ** -16)   # stored in two bf16 parts
