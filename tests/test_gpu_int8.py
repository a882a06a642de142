"""moe_quant_i8, moe_pack_i8 and moe_gemm_i8: codes, scales and the packed layout bit for bit, the
product against exact integer sums in float64 with one rounding to bf16 and the few fp32 roundings
counted in _layer_ref.gemm_i8."""
import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu


def make(T, N, K, seed=0, act=None, add=False):
    g = torch.Generator().manual_seed(seed * 101 + T * 13 + N * 7 + K)
    codes = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int32).to(torch.int8)   # noqa: E731
    c = {"a": codes(T, K), "w": codes(N, K), "sa": torch.rand(T, generator=g) / 64 + 1e-3,
         "sw": (torch.rand(N, generator=g) + 0.1) / (64 * K ** 0.5)}
    No = N // 2 if act else N
    c["add"] = torch.randn(T, No, generator=g).to(torch.bfloat16) if add else None
    return c


def check(T, N, K, act=None, add=False, seed=0, c=None):
    c = c or make(T, N, K, seed, act, add)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    kw = dict(beta=4.0, linear_beta=25.0) if act == "situv2" else {}
    guard = torch.full((T + 2, N // 2 if act else N), 7.0, dtype=torch.bfloat16, device="cuda")
    out = qm.moe_gemm_i8(d["a"], d["sa"], qm.moe_pack_i8(d["w"]), d["sw"], act=act, add=d["add"], out=guard[1:-1], **kw)
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    want, err = ref.gemm_i8(c["a"], c["sa"], c["w"], c["sw"], act, add=c["add"])
    bad = (ref.f64(out) - want).abs() > ref.HALF_BF16 * want.abs() + 1.01 * err + 1e-37
    assert not bad.any(), (T, N, K, act, int(bad.sum()), bad.nonzero()[:4].tolist())
    return out


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 200, 256, 257])
@pytest.mark.parametrize("N,K", [(64, 128), (100, 112), (272, 1456)])
def test_tokens(T, N, K):
    check(T, N, K)


@pytest.mark.parametrize("N", [1, 3, 15, 16, 17, 127, 129, 255, 257, 1000])
@pytest.mark.parametrize("T", [1, 20, 50, 130])
def test_channels(N, T):
    check(T, N, 192, add=True)


@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 128, 144, 256, 1040, 4096])
@pytest.mark.parametrize("T", [1, 40, 140])
def test_depths(K, T):
    check(T, 96, K)


@pytest.mark.parametrize("act", ["situv2", "silu"])
@pytest.mark.parametrize("T,N,K", [(1, 32, 16), (1, 7168, 512), (5, 96, 320), (33, 160, 128), (64, 512, 256), (65, 224, 240),
                                   (300, 544, 384)])
def test_activations(act, T, N, K):
    check(T, N, K, act)
    check(T, N, K, act, add=True)


@pytest.mark.parametrize("T,N,K,act", [(3500, 3584, 272, None), (4000, 3616, 144, "silu"), (3329, 4100, 128, None)])
def test_large_tiles(T, N, K, act):
    check(T, N, K, act, add=act is None)


# (tokens, channels) of every tile shape the sizes choose between: 32 x 64 and 64 x 64 with K in groups,
# 64 x 64, 128 x 128, 256 x 256 in halves, in halves with a half past the tokens, and full ones
# before halves
SHAPES = [(40, 200), (100, 3000), (300, 4000), (700, 4000), (1200, 4100), (1100, 4096), (4300, 4100)]


@pytest.mark.parametrize("K", [16, 80, 128, 272, 400])
@pytest.mark.parametrize("T,N", SHAPES)
def test_tile_shapes(T, N, K):
    check(T, N, K, add=K == 272)


@pytest.mark.parametrize("N", [96, 129, 258, 1004])
@pytest.mark.parametrize("off", [0, 1, 2, 5])
@pytest.mark.parametrize("T", [9, 50, 700])
def test_rows_at_any_address(T, N, off):
    # out and add start at any element: neither their start nor their rows are aligned
    c = make(T, N, 144, add=True)
    buf = torch.full((T * N + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    add = torch.empty(T * N + 16, dtype=torch.bfloat16, device="cuda")[off:off + T * N].view(T, N)
    add.copy_(c["add"])
    out = buf[8 - off:8 - off + T * N].view(T, N)
    qm.moe_gemm_i8(c["a"].cuda(), c["sa"].cuda(), qm.moe_pack_i8(c["w"].cuda()), c["sw"].cuda(), add=add, out=out)
    assert (buf[:8 - off] == 7).all() and (buf[8 - off + T * N:] == 7).all()
    want, err = ref.gemm_i8(c["a"], c["sa"], c["w"], c["sw"], add=c["add"])
    assert not ((ref.f64(out) - want).abs() > ref.HALF_BF16 * want.abs() + 1.01 * err + 1e-37).any()


@pytest.mark.parametrize("K", [16, 144, 528])
@pytest.mark.parametrize("T,N", SHAPES)
@pytest.mark.parametrize("act", ["situv2", "silu"])
def test_tile_shapes_with_activations(act, T, N, K):
    check(T, (N + 31) // 32 * 32, K, act, add=K == 144)


def test_sums_at_the_limits_of_int32():
    # all codes -128: 128 * 128 * K is the largest sum, just below 2^31
    K = (1 << 17) - 16
    for T in (1, 70):
        c = make(T, 20, K)
        c["a"].fill_(-128)
        c["w"].fill_(-128)
        c["w"][1].fill_(127)
        check(T, 20, K, c=c)


def test_add_in_place_equals_add():
    c = make(90, 200, 320, add=True)
    d = {k: v.cuda() for k, v in c.items()}
    p = qm.moe_pack_i8(d["w"])
    want = qm.moe_gemm_i8(d["a"], d["sa"], p, d["sw"], add=d["add"])
    out = d["add"].clone()
    qm.moe_gemm_i8(d["a"], d["sa"], p, d["sw"], add=out, out=out)
    assert torch.equal(out, want)


def test_a_token_does_not_depend_on_its_batch():
    # integer sums: the same bits from the kernel for few tokens and from the one for many
    c = make(260, 544, 400)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    p = qm.moe_pack_i8(d["w"])
    full = qm.moe_gemm_i8(d["a"], d["sa"], p, d["sw"])
    for n in (1, 16, 17, 64, 65, 130):
        assert torch.equal(qm.moe_gemm_i8(d["a"][:n].clone(), d["sa"][:n].clone(), p, d["sw"]), full[:n])


@pytest.mark.parametrize("N,K", [(1, 16), (16, 64), (33, 144), (100, 1456), (256, 128)])
def test_packed_layout(N, K):
    w = make(1, N, K)["w"]
    p = qm.moe_pack_i8(w.cuda()).cpu()
    F, S, _ = p.shape
    full = torch.zeros(F * 16, S * 64, dtype=torch.int8)
    full[:N, :K] = w
    want = full.view(F, 16, S, 4, 16).permute(0, 2, 3, 1, 4).reshape(F, S, 1024)
    assert torch.equal(p, want)


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 512), (5, 528), (9, 3584), (2, 8192), (3, 16400), (2, 40000)])
def test_quant(rows, cols):
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).to(torch.bfloat16)
    q, s = qm.moe_quant_i8(x.cuda())
    wq, ws = ref.quant_i8(x)
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), ws)


def test_quant_edges():
    x = torch.zeros(7, 64, dtype=torch.bfloat16)
    x[1, 3], x[2, 5] = 1e-38, 2.0 ** -100
    x[3] = torch.linspace(-127, 127, 64)
    x[3, 0] = -127.0
    x[4, 1], x[5, 1], x[5, 2] = float("inf"), float("nan"), 3.0
    x[6] = torch.arange(64) - 31.5
    x[6, 0] = 127.0                                            # scale 1: ties to even
    q, s = qm.moe_quant_i8(x.cuda())
    keep = [0, 1, 2, 3, 6]
    wq, ws = ref.quant_i8(x[keep])
    assert torch.equal(q.cpu()[keep], wq) and torch.equal(s.cpu()[keep], ws)
    assert torch.isnan(s[[4, 5]]).all() and (q[[4, 5]] == 0).all()
    assert (q[[0, 1]] == 0).all() and (s[[0, 1]] == 0).all()


@pytest.mark.parametrize("T", [3, 40, 700])
@pytest.mark.parametrize("small", ["gate", "up", "both"])
def test_situv2_of_small_values(T, small):
    # tanh(x) near 0 is x: a quotient through 1 - exp(-2x) would lose what exp rounds away, 1% at x = 5e-6.
    # Besides the rounding to bf16 each tanh may be off by 2^-15 of itself (its worst is where the
    # exponential takes over: a last place of 2^-24 beside 1 - exp = 2^-7.5), the scales' products and the
    # rest by 32 roundings of fp32.
    N, K = 256, 16
    g = torch.Generator().manual_seed(T)
    size = lambda n, on: torch.exp2(-24 * torch.rand(n, generator=g)) if on else 0.5 + torch.rand(n, generator=g)   # noqa: E731
    sw = torch.cat((size(N // 2, small != "up"), size(N // 2, small != "gate")))
    a = torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int32).to(torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int32).to(torch.int8)
    sa = (0.5 + torch.rand(T, generator=g)) / 127 ** 2
    out = qm.moe_gemm_i8(a.cuda(), sa.cuda(), qm.moe_pack_i8(w.cuda()), sw.cuda(), act="situv2", beta=4.0, linear_beta=25.0)
    r = (ref.f64(a) @ ref.f64(w).t()) * ref.f64(sa)[:, None] * ref.f64(sw)
    gate, up = r[:, :N // 2], r[:, N // 2:]
    want = 4.0 * torch.tanh(gate / 4.0) * torch.sigmoid(gate) * 25.0 * torch.tanh(up / 25.0)
    bad = (ref.f64(out) - want).abs() > (ref.HALF_BF16 + 2 * 2.0 ** -15 + 32 * ref.HALF_F32 * (1 + gate.abs())) * want.abs()
    assert not bad.any(), (int(bad.sum()), gate[bad][:4].tolist(), up[bad][:4].tolist())


# a wave's share of K: less than one trip of eight blocks, just one, one and a part, several and a part
@pytest.mark.parametrize("K", [448, 512, 528, 3584, 3600, 4080, 4096, 4112, 4608, 7168, 8192, 8208, 12304])
def test_depths_of_few_tokens(K):
    for T, act in ((1, None), (16, "silu"), (7, "situv2")):
        check(T, 96, K, act, add=act is None)
