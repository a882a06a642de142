"""Microscaled codes (rows, transposes, packed, stochastic) bit for bit, and the MXFP4 product: exact where
its sums are, else within the bound of its fp32 sums."""
import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def matrix(R, C, dt, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * R + C)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-20, 20, (R, C), generator=g) * (torch.rand(R, C, generator=g) < 0.1))
    x = x * torch.exp2(torch.randint(-12, 12, (R, 1), generator=g).float())
    x[torch.rand(R, C, generator=g) < 0.05] = 0.0
    x[0, : min(C, 40)] = -0.0
    return x.to(TYPES[dt]), torch.randint(0, 256, (R, C), generator=g, dtype=torch.int32).to(torch.uint8)


def flat(q, kind):
    return ref.unpairs(q.cpu()) if kind == "fp4" else q.cpu()


def check_codes(q, s, x, kind, packed, noise):
    want, ws = ref.mx_codes(x, kind, noise)
    if packed:
        want, ws = ref.mx_packed(ref.pairs(want), ws)
        # what fills the rows up to 16 is zero
        assert torch.equal(q.cpu(), want) and torch.equal(s.cpu(), ws)
    else:
        assert torch.equal(s.cpu(), ws)
        got = flat(q, kind)
        assert torch.equal(got, want), (got != want).nonzero()[:4]


SIZES = [(1, 3584), (1, 1), (7, 31), (33, 129), (128, 64), (130, 257), (300, 100), (64, 1790), (16, 4096)]


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("noisy", [False, True])
def test_codes(R, C, dt, noisy):
    x, noise = matrix(R, C, dt)
    nz = noise if noisy else None
    xd, nd = x.cuda(), noise.cuda() if noisy else None
    nt = None if nz is None else nz.t()
    for kind in ("fp8", "fp4"):
        r = qm.moe_quant_mx(xd, kind, noise=nd)
        assert r.t is None
        check_codes(r.q, r.q_scale, x, kind, False, nz)
        r = qm.moe_quant_mx(xd, t_dtype=kind, noise=nd)
        assert r.q is None
        check_codes(r.t, r.t_scale, x.t(), kind, False, nt)
    r = qm.moe_quant_mx(xd, "fp4", packed=True, noise=nd)
    check_codes(r.q, r.q_scale, x, "fp4", True, nz)
    r = qm.moe_quant_mx(xd, "fp8", t_dtype="fp4", t_packed=True, noise=nd)
    check_codes(r.q, r.q_scale, x, "fp8", False, nz)
    check_codes(r.t, r.t_scale, x.t(), "fp4", True, nt)
    r = qm.moe_quant_mx(xd, "fp4", packed=True, t_dtype="fp8", noise=nd)
    check_codes(r.q, r.q_scale, x, "fp4", True, nz)
    check_codes(r.t, r.t_scale, x.t(), "fp8", False, nt)


def test_same_codes_as_quant_act():
    x = matrix(50, 256, "bf16")[0].cuda()
    for kind in ("fp8", "fp4"):
        q, s = qm.moe_quant_act(x, kind)
        r = qm.moe_quant_mx(x, kind)
        assert torch.equal(r.q, q) and torch.equal(r.q_scale, s)


def test_extreme_values():
    # the smallest and largest fp32 values, ties, saturated ones, and blocks with Inf and NaN
    x = torch.zeros(8, 160)
    x[0, :32] = 2.0 ** -149 * torch.arange(32)
    x[1, :32] = torch.finfo(torch.float32).max * torch.linspace(-1, 1, 32)
    x[2, :64] = torch.linspace(-6, 6, 64)
    x[3, :33] = torch.arange(33) * 0.25                        # ties of both grids
    x[4, 40] = float("inf")
    x[5, 70] = float("nan")
    x[6] = torch.linspace(-511, 511, 160)
    x[7] = 2.0 ** -126
    for noise in (None, torch.full((8, 160), 255, dtype=torch.uint8), torch.zeros(8, 160, dtype=torch.uint8)):
        nd = None if noise is None else noise.cuda()
        nt = None if noise is None else noise.t()
        for kind in ("fp8", "fp4"):
            r = qm.moe_quant_mx(x.cuda(), kind, t_dtype=kind, noise=nd)
            check_codes(r.q, r.q_scale, x, kind, False, noise)
            check_codes(r.t, r.t_scale, x.t(), kind, False, nt)


def test_stochastic_mean():
    # over all 256 noise values the mean is the value, to 1/512 of a step and what the sum of 256 exact terms adds
    v = torch.rand(32, generator=torch.Generator().manual_seed(3)) * 6
    v[0] = 6.0
    x = v[None].repeat(256, 1)
    noise = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 32)
    r = qm.moe_quant_mx(x.cuda(), "fp4", noise=noise.cuda())
    got = ref.mx_values(flat(r.q, "fp4"), r.q_scale.cpu(), "fp4")[:, :32].mean(0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    assert ((got - v.double()).abs() <= step / 512 + 1e-12).all()


@pytest.mark.parametrize("N,K", [(1, 32), (16, 128), (33, 160), (100, 3584), (257, 96)])
def test_pack(N, K):
    g = torch.Generator().manual_seed(N + K)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    s = torch.randint(100, 140, (N, K // 32), generator=g, dtype=torch.int32).to(torch.uint8)
    kp = (K + 127) // 128 * 128
    wf, sf = torch.zeros(N, kp // 2, dtype=torch.uint8), torch.zeros(N, kp // 32, dtype=torch.uint8)
    wf[:, : K // 2], sf[:, : K // 32] = w, s
    q, qs = qm.moe_pack_mx(w.cuda(), s.cuda())
    want, ws = ref.mx_packed(wf, sf)
    assert torch.equal(q.cpu(), want) and torch.equal(qs.cpu(), ws)


def operands(T, N, K, kind, spread, seed=0):
    """Codes whose values are whole multiples of 2^-spread / 2: with the scales in [2^-spread, 1] and K columns
    every partial sum is a multiple of 2^(-2 spread - 2) below 36 K, so fp32 holds it exactly for
    36 K 2^(2 spread + 2) < 2^24 (fp8 elements are taken up to 6 in steps of 1/2, as fp4's)."""
    g = torch.Generator().manual_seed(seed + T + 3 * N + 7 * K)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.int32).to(torch.uint8)   # noqa: E731
    a = r(0, 16, T, K)
    va = ref.E2M1[(a & 7).long()] * (1 - 2 * (a >> 3).double())
    if kind == "fp8":
        a = va.float().to(torch.float8_e4m3fn).view(torch.uint8)
    w = r(0, 16, N, K)
    sa, sw = r(127 - spread, 128, T, K // 32), r(127 - spread, 128, N, K // 32)
    return a, sa, w, sw


def exact_product(a, sa, w, sw, kind):
    return ref.mx_values(a.cuda(), sa.cuda(), kind) @ ref.mx_values(w.cuda(), sw.cuda(), "fp4").t()


def product(a, sa, w, sw, kind, **kw):
    ad = (ref.pairs(a) if kind == "fp4" else a).contiguous().cuda()
    p, ps = qm.moe_pack_mx(ref.pairs(w).cuda(), sw.cuda())
    return qm.moe_gemm_mx(ad, sa.cuda(), kind, p, ps, w.shape[0], **kw)


def eights(a, b):
    """What the matrix instruction drops of fp8 tokens' products: it adds those of columns 8 i .. 8 i + 7 in
    fixed point down to 2^-13 of the largest one's power of two, so each of the seven others loses less than
    2^-13 of the largest."""
    fill = -a.shape[1] % 8
    a, b = (torch.nn.functional.pad(m.abs(), (0, fill)) for m in (a, b))
    total = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for i in range(0, a.shape[1], 8):
        top = torch.zeros_like(total)
        for j in range(i, i + 8):
            top = torch.maximum(top, a[:, j, None] * b[None, :, j])
        total += top
    return 7 * 2.0 ** -13 * total


# from streamed weights to the largest tiles; odd numbers of K steps, of tokens and of channels
SHAPES = [(1, 16, 128), (1, 1000, 640), (2, 5000, 128), (3, 77, 3584), (9, 5000, 640), (16, 300, 1152), (16, 64, 2304), (17, 64, 128), (33, 100, 640), (64, 7168, 256),
          (100, 333, 896), (250, 2600, 640), (256, 3584, 384), (900, 2100, 640), (1000, 2048, 256), (2100, 2130, 384),
          (2049, 4100, 640)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_product_exact(T, N, K, kind):
    a, sa, w, sw = operands(T, N, K, kind, 2 if K < 1700 else 1)
    want = exact_product(a, sa, w, sw, kind)
    got = product(a, sa, w, sw, kind, out_dtype=torch.float32)
    assert torch.equal(got.double(), want), (got.double() != want).nonzero()[:5]
    assert torch.equal(product(a, sa, w, sw, kind), want.bfloat16())
    add = torch.randint(-8, 8, (T, N), generator=torch.Generator().manual_seed(1)).float().cuda()
    got = product(a, sa, w, sw, kind, add=add, out_dtype=torch.float32)
    assert torch.equal(got.double(), want + add.double())
    into = add.bfloat16()
    out = product(a, sa, w, sw, kind, add=into, out=into)      # summed in place
    assert out.data_ptr() == into.data_ptr() and torch.equal(out, (want + add.double()).bfloat16())


@pytest.mark.parametrize("T,N,K", [(1, 32, 128), (5, 416, 640), (16, 7168, 384), (40, 224, 640), (250, 2592, 384), (600, 2080, 640),
                                   (900, 2112, 640), (2100, 2144, 256), (2049, 4128, 384)])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("act", ["situv2", "silu"])
def test_product_activated(T, N, K, kind, act):
    a, sa, w, sw = operands(T, N, K, kind, 2)
    sw -= 6                                                    # sums of a few units
    r = exact_product(a, sa, w, sw, kind)
    want = ref.activated(r, act)
    kw = dict(beta=4.0, linear_beta=25.0) if act == "situv2" else {}
    got = product(a, sa, w, sw, kind, act=act, out_dtype=torch.float32, **kw).double()
    # r is exact; exponentials, quotients and products of the activation: a few steps each, of fast sigmoids
    # whose exponent's rounding weighs |g|
    g, u = r.chunk(2, 1)
    err = 32 * ref.HALF_F32 * (1 + g.abs()) * want.abs()
    if act == "situv2":
        err = err + 32 * ref.HALF_F32 * 100 * torch.sigmoid(g) * (torch.tanh(g / 4).abs() + torch.tanh(u / 25).abs()) * 2.0 ** -7
        err = err + 2.0 ** -16 * want.abs()                    # the series of 1 - exp next to 0
    assert ((got - want).abs() <= err).all(), float(((got - want).abs() - err).max())
    add = torch.ones(T, N // 2, device="cuda", dtype=torch.bfloat16)
    b = product(a, sa, w, sw, kind, act=act, add=add, **kw).double()
    assert ((b - want - 1).abs() <= ref.HALF_BF16 * (want + 1).abs() + 1.01 * err + ref.HALF_F32 * (want.abs() + 1)).all()


@pytest.mark.parametrize("T,N,K", [(1, 500, 3584), (60, 500, 1000), (700, 1000, 1790)])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_linear_layer_and_its_gradients(T, N, K, kind):
    # forward and both gradients from coded matrices, against float64 products of the values of the codes
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, K, generator=g), torch.randn(N, K, generator=g) / K ** 0.5
    dy, noise = torch.randn(T, N, generator=g).bfloat16(), torch.randint(0, 256, (T, N), generator=g, dtype=torch.int32).to(torch.uint8)
    val = lambda m, k, n=None: ref.mx_values(*ref.mx_codes(m, k, n), k)[:, : m.shape[1]].cuda()   # noqa: E731
    xq = qm.moe_quant_mx(x.cuda(), kind, t_dtype="fp4", t_packed=True)
    wq = qm.moe_quant_mx(w.cuda(), "fp4", packed=True, t_dtype="fp4", t_packed=True)
    dq = qm.moe_quant_mx(dy.cuda(), kind, t_dtype=kind, noise=noise.cuda())
    steps = lambda k: 2 * ref.HALF_F32 * (k / 32 + 16)   # noqa: E731  # roundings of the fp32 sums, of 32 columns each at the finest

    def close(got, a, b, half):
        want, mag = a @ b.t(), a.abs() @ b.abs().t()
        err = half * want.abs() + steps(a.shape[1]) * mag
        if kind == "fp8" and got.dtype == torch.bfloat16:
            err = err + eights(a, b)
        assert ((got.double() - want).abs() <= err).all()
    close(qm.moe_gemm_mx(xq.q, xq.q_scale, kind, wq.q, wq.q_scale, N), val(x, kind), val(w, "fp4"), ref.HALF_BF16)
    close(qm.moe_gemm_mx(dq.q, dq.q_scale, kind, wq.t, wq.t_scale, K), val(dy, kind, noise), val(w.t(), "fp4"), ref.HALF_BF16)
    dw = qm.moe_gemm_mx(dq.t, dq.t_scale, kind, xq.t, xq.t_scale, K, out_dtype=torch.float32)
    close(dw, val(dy.t(), kind, noise.t()), val(x.t(), "fp4"), ref.HALF_F32)
    # accumulated over two batches, in place
    two = qm.moe_gemm_mx(dq.t, dq.t_scale, kind, xq.t, xq.t_scale, K, add=dw, out=dw.clone())
    assert torch.equal(two, 2 * dw)
    # the products are linear: a difference of outputs along dX is the product's own (exact in its values)
    assert dw.shape == (N, K)


@pytest.mark.parametrize("T", [2, 40, 2100])
def test_bad_blocks_reach_their_row_and_channel_only(T):
    x, w = torch.randn(T, 256), torch.randn(2144, 256)
    x[1, 200], w[5, 3] = float("inf"), float("nan")
    for kind in ("fp8", "fp4"):
        a = qm.moe_quant_mx(x.cuda(), kind)
        b = qm.moe_quant_mx(w.cuda(), "fp4", packed=True)
        bad = qm.moe_gemm_mx(a.q, a.q_scale, kind, b.q, b.q_scale, 2144).isnan()
        want = torch.zeros_like(bad)
        want[1], want[:, 5] = True, True
        assert torch.equal(bad, want)


def test_rows_behind_the_last_stay():
    out = torch.full((40, 96), 5.0, device="cuda", dtype=torch.bfloat16)
    a, sa, w, sw = operands(33, 96, 256, "fp4", 1)
    product(a, sa, w, sw, "fp4", out=out[:33])
    assert (out[33:] == 5.0).all() and torch.equal(out[:33], exact_product(a, sa, w, sw, "fp4").bfloat16())


def test_unaligned_outputs():
    # rows of 101 channels in a buffer that starts at an odd element
    a, sa, w, sw = operands(50, 101, 256, "fp8", 1)
    store = torch.zeros(50 * 101 + 1, device="cuda", dtype=torch.bfloat16)
    out = store[1:].view(50, 101)
    product(a, sa, w, sw, "fp8", out=out)
    assert torch.equal(out, exact_product(a, sa, w, sw, "fp8").bfloat16()) and store[0] == 0


def test_norm_codes_feed_the_product():
    # codes of both norms are operands of the product as they are
    x = torch.randn(20, 384, device="cuda")
    w = qm.moe_quant_mx(torch.randn(64, 384, device="cuda"), "fp4", packed=True)
    ones = torch.ones(384, device="cuda")
    for kind in ("fp8", "fp4"):
        for r in (qm.moe_layer_norm(x, w=ones, q_dtype=kind), qm.moe_block_norm(x, w_pre=ones, q_dtype=kind)):
            got = qm.moe_gemm_mx(r.q, r.q_scale, kind, w.q, w.q_scale, 64, out_dtype=torch.float32).double()
            codes = ref.unpairs(r.q) if kind == "fp4" else r.q
            va = ref.mx_values(codes, r.q_scale, kind)
            f, s, _ = w.q.shape
            wv = w.q.view(f, s, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(f * 16, -1)
            ws = w.q_scale.view(f, s, 16, 4).permute(0, 2, 1, 3).reshape(f * 16, -1)
            vw = ref.mx_values(ref.unpairs(wv), ws, "fp4")
            want, mag = va @ vw.t(), va.abs() @ vw.abs().t()
            assert ((got - want).abs() <= 2 * ref.HALF_F32 * 28 * mag).all()
