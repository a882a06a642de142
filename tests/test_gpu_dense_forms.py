"""Calls that the documentation allows, of the operators beside the routed experts, at sizes and addresses where a
kernel takes another way: coded norms of every width, rows and matrices at odd addresses, one expert, wide
intermediates, results and gradients of which only some are asked for."""
import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu


def at_odd_element(t):
    """The same tensor one element into a buffer."""
    store = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    store[1:] = t.flatten()
    return store[1:].view(t.shape)


@pytest.mark.parametrize("D", [32, 64, 480, 512, 544, 3584, 8192, 8224, 12000, 16384])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["fp8", "fp4", "i8"])
def test_coded_norms(D, dt, kind):
    T = 9
    g = torch.Generator().manual_seed(D)
    x, y = (2 * torch.randn(T, D, generator=g)).to(dt), torch.randn(T, D, generator=g).bfloat16()
    w, b = 1 + 0.2 * torch.randn(D, generator=g), 0.3 * torch.randn(D, generator=g)
    x[4] = 0
    y[4] = 0                                                   # its codes are those of the bias
    r = qm.moe_layer_norm(x.cuda(), y.cuda(), w=w.cuda(), b=b.cuda(), q_dtype=kind)
    h = x.double() + y.double()
    n = ref.layer_norm(h, None, w.double(), b.double(), 1e-5)[1]
    _, _, z, ez = ref.layer_norm_parts(h, 1e-5)
    err = 1.01 * (ez * w.abs() + 2 * ref.HALF_F32 * ((z * w).abs() + b.abs()))
    assert ((r.n.cpu().double() - n).abs() <= ref.HALF_BF16 * n.abs() + err).all()
    if kind == "i8":
        s = r.q_scale.cpu().double()[:, None]
        amax = n.abs().amax(1, keepdim=True)
        assert ((s * 127 - amax).abs() <= err.amax(1, keepdim=True) + 4 * ref.HALF_F32 * amax).all()
        # half a code, and what the value and the quotient are off by (codes up to 127: 4 steps of them)
        assert ((r.q.cpu().double() * s - n).abs() <= s * (0.5 + 127 * 8 * ref.HALF_F32) + err).all()
        return
    codes = ref.unpairs(r.q.cpu()) if kind == "fp4" else r.q.cpu()
    got = ref.mx_values(codes, r.q_scale.cpu(), kind)
    value = lambda v: ref.mx_values(*ref.mx_codes(v, kind), kind)[:, :D]   # noqa: E731
    # the codes of n, or of what its error reaches: on the other side of a border of its own, or with the
    # scale on the other side of a power of two
    near = torch.stack([value(v) for v in (n, n + err, n - err, n + err * n.sign(), n - err * n.sign())])
    assert (got <= near.amax(0)).all() and (got >= near.amin(0)).all()
    assert (got == near[0]).double().mean() > 0.99


@pytest.mark.parametrize("D", [1, 7, 200, 1790, 9001])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_norm_at_odd_addresses(D, dt):
    T = 11
    g = torch.Generator().manual_seed(D)
    n = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    t = dict(x=n(T, D).to(dt), y=n(T, D).bfloat16(), w=n(D), b=n(D), dh=n(T, D).to(dt), dn=n(T, D).bfloat16())
    o = {k: at_odd_element(v) for k, v in t.items()}

    def both(t):
        r = qm.moe_layer_norm(t["x"], t["y"], w=t["w"], b=t["b"], stats=True)
        return r, qm.moe_layer_norm_backward(t["x"], t["y"], r.stats, t["dh"], t["dn"], w=t["w"])
    for a, b in zip(both(t), both(o)):
        for k, v in a._asdict().items():
            assert (v is None) == (getattr(b, k) is None) and (v is None or torch.equal(v, getattr(b, k))), k


@pytest.mark.parametrize("D", [96, 777, 9000])
def test_some_of_the_gradients(D):
    T = 300
    g = torch.Generator().manual_seed(D)
    n = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    x, w, b, dn = n(T, D), n(D), n(D), n(T, D).bfloat16()
    st = qm.moe_layer_norm(x, w=w, b=b, stats=True).stats
    full = qm.moe_layer_norm_backward(x, None, st, None, dn, w=w)
    no_b = qm.moe_layer_norm_backward(x, None, st, None, dn, w=w, bias=False)
    assert torch.equal(no_b.dx, full.dx) and torch.equal(no_b.dw, full.dw) and no_b.db is None
    ones = qm.moe_layer_norm_backward(x, None, st, None, dn, w=torch.ones_like(w))
    none = qm.moe_layer_norm_backward(x, None, st, None, dn, bias=False)
    only_b = qm.moe_layer_norm_backward(x, None, st, None, dn)
    for r in (none, only_b):
        assert torch.equal(r.dx, ones.dx) and r.dw is None
    assert none.db is None and torch.equal(only_b.db, ones.db)


@pytest.mark.parametrize("R,C", [(1, 33), (130, 257), (300, 100), (128, 192)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_coding_at_odd_addresses(R, C, dt):
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C, generator=g).to(dt).cuda()
    noise = torch.randint(0, 256, (R, C), generator=g, dtype=torch.int32).to(torch.uint8).cuda()
    for nz in (None, noise):
        for kw in (dict(q_dtype="fp8"), dict(q_dtype="fp4", t_dtype="fp8"), dict(t_dtype="fp4", t_packed=True)):
            a = qm.moe_quant_mx(x, noise=nz, **kw)
            b = qm.moe_quant_mx(at_odd_element(x), noise=None if nz is None else at_odd_element(nz), **kw)
            for u, v in zip(a, b):
                assert (u is None and v is None) or torch.equal(u, v)


@pytest.mark.parametrize("T,N,K", [(3, 96, 512), (40, 96, 512), (700, 2080, 256)])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_product_with_addend_in_place(T, N, K, kind):
    # every type of result, with an activation, the addend where the result goes, both at an odd element
    g = torch.Generator().manual_seed(T)
    a = qm.moe_quant_mx(torch.randn(T, K, generator=g).cuda(), kind)
    w = qm.moe_quant_mx(torch.randn(N, K, generator=g).cuda() / K ** 0.5, "fp4", packed=True)
    for act, kw in ((None, {}), ("silu", {}), ("situv2", dict(beta=4.0, linear_beta=25.0))):
        for dt in (torch.bfloat16, torch.float32):
            add = torch.randn(T, N if act is None else N // 2, generator=g).to(dt).cuda()
            want = qm.moe_gemm_mx(a.q, a.q_scale, kind, w.q, w.q_scale, N, act=act, add=add, out_dtype=dt, **kw)
            into = at_odd_element(add)
            got = qm.moe_gemm_mx(a.q, a.q_scale, kind, w.q, w.q_scale, N, act=act, add=into, out=into, **kw)
            assert got.data_ptr() == into.data_ptr() and torch.equal(got, want)


def experts(E, D, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)   # noqa: E731
    e = lambda *s: torch.randint(118, 121, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)   # noqa: E731
    return qm.moe_pack_w1(b(E, 2 * I, D // 2)), e(E, 2 * I, D // 32), qm.moe_pack_w2(b(E, D, I // 2)), e(E, D, I // 32)


@pytest.mark.parametrize("a", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,E,K,D,I", [(1, 1, 1, 128, 128), (16, 1, 1, 128, 128), (2, 3, 2, 128, 8192), (16, 6, 3, 256, 8192), (3, 4, 2, 8192, 128),
                                       (12, 4, 4, 8192, 128)])
def test_few_tokens_of_other_shapes(a, T, E, K, D, I):
    w = experts(E, D, I, T + D)
    g = torch.Generator().manual_seed(T)
    x, xs = torch.randn(T, D, generator=g).bfloat16().cuda(), None
    if a != "bf16":
        x, xs = qm.moe_quant_act(x, a)
    l = torch.randn(T, E, generator=g).cuda()
    for act, kw in (("silu", {}), ("situv2", dict(beta=4.0, linear_beta=25.0))):
        r = qm.moe_routed_few(l, x, xs, a, *w, K, act=act, **kw)
        c = qm.moe_router(l, K)
        lay = qm.moe_sort(c.ids, c.w, 0, E, 16)
        want = qm.moe_fused(x, xs, a, *w, c.w, lay, E, act, kw.get("beta"), kw.get("linear_beta")).double()
        assert torch.equal(r.ids, c.ids) and ((r.w - c.w).abs() <= 1e-5 * c.w).all()
        # moe_fused rounds the intermediate (bf16) and each weighted row; codes of the intermediate may differ at borders:
        # the 2-norm of K I roundings that average out, each at most 2^-8 of its term, and of the outputs'
        assert float((r.out.double() - want).norm() / want.norm()) < 2.0 ** -7


@pytest.mark.parametrize("T", [2, 12])
def test_few_tokens_none_valid_or_local(T):
    w = experts(8, 128, 128, 5)
    x, l = torch.randn(T, 128, device="cuda").bfloat16(), torch.randn(T, 64, device="cuda")
    kw = dict(beta=4.0, linear_beta=25.0)
    r = qm.moe_routed_few(l, x, None, "bf16", *w, 4, valid=torch.zeros(T, dtype=torch.bool, device="cuda"), **kw)
    assert (r.out == 0).all() and (r.ids == -1).all() and (r.w == 0).all()
    for begin in (64, 2 ** 31 - 8, -8, -2 ** 31):
        r = qm.moe_routed_few(l, x, None, "bf16", *w, 4, expert_begin=begin, **kw)
        assert (r.out == 0).all() and (r.ids >= 0).all()
