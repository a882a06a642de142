"""Layer norm, the MXFP4 products and the routed layer of a few tokens together, as a program runs them: a
decode step and a training step, eager, in HIP graphs that are replayed with new inputs while others live,
on another stream, and on two streams at once, every time with the bits of the eager run; and sizes past
2^31 elements and past one dispatch."""
import pytest
import torch

import _dense_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
D, E, K, I, F = 384, 24, 4, 128, 320
SITU = dict(act="situv2", beta=4.0, linear_beta=25.0)


@pytest.fixture(scope="module")
def weights():
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    b = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)   # noqa: E731
    e = lambda *s: torch.randint(118, 121, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)   # noqa: E731
    return {"w": 1 + 0.1 * n(D), "b": 0.1 * n(D), "router": n(E, D) / D ** 0.5,
            "up": qm.moe_pack_mx(b(2 * F, D // 2), e(2 * F, D // 32)), "down": qm.moe_pack_mx(b(D, F // 2), e(D, F // 32)),
            "experts": (qm.moe_pack_w1(b(E, 2 * I, D // 2)), e(E, 2 * I, D // 32), qm.moe_pack_w2(b(E, D, I // 2)), e(E, D, I // 32))}


def decode_inputs(T, seed=0):
    g = torch.Generator().manual_seed(50 * seed + T)
    return {"x": (2 * torch.randn(T, D, generator=g)).cuda(), "y": torch.randn(T, D, generator=g).bfloat16().cuda()}


def decode(w, s):
    """Residual sum and norm, the routed experts and a dense MXFP4 block beside them, the next norm."""
    o = {}
    a = qm.moe_layer_norm(s["x"], s["y"], w=w["w"], b=w["b"], q_dtype="fp8")
    o.update(h=a.h, n=a.n, q=a.q, qs=a.q_scale)
    r = qm.moe_routed_few(a.n.float() @ w["router"].t(), a.q, a.q_scale, "fp8", *w["experts"], K, **SITU)
    o.update(routed=r.out, ids=r.ids, rw=r.w)
    o["mid"] = qm.moe_gemm_mx(a.q, a.q_scale, "fp8", *w["up"], 2 * F, **SITU)
    m = qm.moe_quant_mx(o["mid"], "fp4")
    o.update(mq=m.q, ms=m.q_scale)
    o["out"] = qm.moe_gemm_mx(m.q, m.q_scale, "fp4", *w["down"], D, add=r.out)
    b = qm.moe_layer_norm(a.h, o["out"], w=w["w"], b=w["b"])
    o.update(h2=b.h, n2=b.n)
    return o


def train_inputs(T, seed=0):
    g = torch.Generator().manual_seed(70 * seed + T)
    n = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    return {"x": n(T, 200), "y": n(T, 200).bfloat16(), "w": n(200), "b": n(200), "W": n(72, 200) / 14, "dy": n(T, 72).bfloat16(),
            "dh": n(T, 200), "noise": torch.randint(0, 256, (T, 72), generator=g, dtype=torch.int32).to(torch.uint8).cuda()}


def train(s):
    """Layer norm and a linear layer in MXFP4, forward and backward."""
    a = qm.moe_layer_norm(s["x"], s["y"], w=s["w"], b=s["b"], stats=True)
    x = qm.moe_quant_mx(a.n, "fp8", t_dtype="fp4", t_packed=True)
    w = qm.moe_quant_mx(s["W"], "fp4", packed=True, t_dtype="fp4", t_packed=True)
    y = qm.moe_gemm_mx(x.q, x.q_scale, "fp8", w.q, w.q_scale, 72)
    d = qm.moe_quant_mx(s["dy"], "fp8", t_dtype="fp4", noise=s["noise"])
    dn = qm.moe_gemm_mx(d.q, d.q_scale, "fp8", w.t, w.t_scale, 200)
    dW = qm.moe_gemm_mx(d.t, d.t_scale, "fp4", x.t, x.t_scale, 200, out_dtype=torch.float32)
    g = qm.moe_layer_norm_backward(s["x"], s["y"], a.stats, s["dh"], dn, w=s["w"])
    return dict(h=a.h, n=a.n, y=y, dn=dn, dW=dW, **g._asdict())


def equal(a, b):
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def captured(fn, s):
    for _ in range(2):                                          # sizes and workspaces settle before the capture
        fn(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn(s)
    return graph, out


def replayed(fn, make, sizes):
    graphs = [(s, *captured(fn, s)) for s in map(make, sizes)]   # all alive at once
    for turn in range(4):
        for s, graph, out in graphs:
            new = make(s["x"].shape[0], seed=turn + 1)
            want = {k: v.clone() for k, v in fn(new).items()}
            for k in s:
                s[k].copy_(new[k])
            graph.replay()
            torch.cuda.synchronize()
            equal(want, out)


def test_decode_in_graphs(weights):
    replayed(lambda s: decode(weights, s), decode_inputs, (1, 3, 16))


def test_training_step_in_graphs():
    replayed(train, train_inputs, (40, 700))


def test_training_step_against_float64():
    s = train_inputs(90)
    o = train(s)
    f = {k: v.double() for k, v in s.items()}
    h, n = ref.layer_norm(f["x"], f["y"], f["w"], f["b"], 1e-5)
    assert ((o["n"].double() - n).abs() <= ref.HALF_BF16 * n.abs() + 1e-5).all()
    # the products, on the GPU's own operands: fp32 sums of the codes' values
    val = lambda m, k, nz=None: ref.mx_values(*ref.mx_codes(m, k, nz), k)[:, : m.shape[1]].cuda()   # noqa: E731
    dW, mag = val(s["dy"].t(), "fp4", s["noise"].t()) @ val(o["n"].t(), "fp4").t(), None
    assert ((o["dW"].double() - dW).abs() <= 1e-5 * dW.abs().max()).all()
    y = val(o["n"], "fp8") @ val(s["W"], "fp4").t()
    assert ((o["y"].double() - y).abs() <= ref.HALF_BF16 * y.abs() + 1e-3 * y.abs().mean()).all()
    # the norm's gradient by autograd, of the GPU's dn
    leaves = [f[k].requires_grad_(True) for k in ("x", "w", "b")]
    h, n = ref.layer_norm(leaves[0], f["y"], leaves[1], leaves[2], 1e-5)
    dx, dw, db = torch.autograd.grad((h, n), leaves, (f["dh"], o["dn"].double()))
    for got, want in ((o["dx"], dx), (o["dw"], dw), (o["db"], db)):
        assert float((got.double() - want).norm() / want.norm()) < 1e-5


def test_on_another_stream(weights):
    s, t = decode_inputs(7), train_inputs(130)
    want, want_t = decode(weights, s), train(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, got_t = decode(weights, s), train(t)
    side.synchronize()
    equal(want, got)
    equal(want_t, got_t)


def test_two_streams_at_once(weights):
    cases = [train_inputs(1500, seed=i) for i in range(2)]
    steps = [decode_inputs(9, seed=i) for i in range(2)]
    want = [{k: v.clone() for k, v in {**train(c), **{"d" + k: v for k, v in decode(weights, s).items()}}.items()}
            for c, s in zip(cases, steps)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = {**train(cases[i]), **{"d" + k: v for k, v in decode(weights, steps[i]).items()}}
    torch.cuda.synchronize()
    for i in range(2):
        equal(want[i], got[i])


def test_rows_past_one_dispatch():
    # 2^27 + 5 rows of one column: codes along the rows (16 work items each, in slices) and of the transpose
    R = 2 ** 27 + 5
    x = (torch.arange(R, device="cuda", dtype=torch.int32) % 7 - 3).bfloat16().view(R, 1)
    r = qm.moe_quant_mx(x, "fp4", t_dtype="fp4")
    small = qm.moe_quant_mx(x[:7].contiguous(), "fp4")
    for name, per in (("q", 64), ("q_scale", 4)):
        full, one = getattr(r, name), getattr(small, name)
        rows = R // 7 * 7
        assert torch.equal(full[:rows].view(-1, 7 * per), one.view(1, 7 * per).expand(rows // 7, 7 * per)), name
        assert torch.equal(full[rows:], one[: R - rows]), name
    only = qm.moe_quant_mx(x, "fp4")                            # the kernel of rows alone
    assert torch.equal(only.q, r.q) and torch.equal(only.q_scale, r.q_scale)
    # the transpose: 224 = 7 * 32 values repeat
    tail = qm.moe_quant_mx(x[:224].contiguous(), t_dtype="fp4")
    whole = R // 224 * 112
    assert torch.equal(r.t[0, :whole].view(-1, 112), tail.t[:, :112].expand(whole // 112, 112))
    assert (r.t[0, (R + 1) // 2:] == 0).all()


def test_norm_rows_past_one_dispatch():
    R = 2 ** 26 + 9
    x = torch.randn(4099, 8, device="cuda").bfloat16().repeat(R // 4099 + 1, 1)[:R].contiguous()
    w, b = torch.rand(8, device="cuda") + 0.5, torch.randn(8, device="cuda")
    r = qm.moe_layer_norm(x, w=w, b=b, stats=True)
    one = qm.moe_layer_norm(x[:4099].contiguous(), w=w, b=b, stats=True)
    whole = R // 4099 * 4099
    assert torch.equal(r.n[:whole].view(-1, 4099 * 8), one.n.view(1, -1).expand(whole // 4099, -1))
    assert torch.equal(r.n[whole:], one.n[: R - whole]) and torch.equal(r.stats[:, whole:], one.stats[:, : R - whole])
    del one
    dn = torch.ones_like(x)
    d = qm.moe_layer_norm_backward(x, None, r.stats, None, dn, w=w)
    assert (d.db == float(R)).all() or ((d.db.double() - R).abs() <= 192 * ref.HALF_F32 * R).all()
    last = qm.moe_layer_norm_backward(x[-600:].contiguous(), None, r.stats[:, -600:].contiguous(), None, dn[:600], w=w)
    assert torch.equal(d.dx[-600:], last.dx)


def test_past_2_31_elements():
    T, D_ = 600_011, 3584
    x = torch.randn(1009, D_, device="cuda").bfloat16().repeat(T // 1009 + 1, 1)[:T].contiguous()
    w, b = torch.rand(D_, device="cuda") + 0.5, torch.randn(D_, device="cuda")
    r = qm.moe_layer_norm(x, w=w, b=b, q_dtype="fp8")
    one = qm.moe_layer_norm(x[-900:].contiguous(), w=w, b=b, q_dtype="fp8")
    assert torch.equal(r.n[-900:], one.n) and torch.equal(r.q[-900:], one.q) and torch.equal(r.q_scale[-900:], one.q_scale)
    q = qm.moe_quant_mx(x, "fp4", t_dtype="fp4")
    o = qm.moe_quant_mx(x[-907:].contiguous(), "fp4")
    assert torch.equal(q.q[-907:], o.q) and torch.equal(q.q_scale[-907:], o.q_scale)
    first = (T - 907) // 32 * 32                                # blocks of 32 rows of the transpose
    o = qm.moe_quant_mx(x[first:].contiguous(), t_dtype="fp4")
    n = q.t.shape[1] - first // 2
    assert torch.equal(q.t[:, first // 2:], o.t[:, :n]) and (o.t[:, n:] == 0).all()


def test_product_past_2_31_outputs():
    T, N = 66_003, 33_000
    w = qm.moe_quant_mx(torch.randn(N, 128, device="cuda"), "fp4", packed=True)
    a = qm.moe_quant_mx(torch.randn(T, 128, device="cuda"), "fp4")
    out = qm.moe_gemm_mx(a.q, a.q_scale, "fp4", w.q, w.q_scale, N)
    for lo in (0, 30_011, T - 300):
        part = qm.moe_gemm_mx(a.q[lo:lo + 300].contiguous(), a.q_scale[lo:lo + 300].contiguous(), "fp4", w.q, w.q_scale, N)
        assert torch.equal(out[lo:lo + 300], part)              # K of 128: one product, whatever the tile


def whole_codes(rows, K, g):
    """fp4x2 codes (any byte) and scales of 1: sums of at most 36 K quarters, exact in fp32 for K up to 2^16."""
    return (torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.full((rows, K // 32), 127, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("T", [3, 20, 300])
def test_weights_past_2_31_bytes(T):
    g = torch.Generator(device="cuda").manual_seed(T)
    N, K_ = 70_000, 65_536
    w = torch.randint(0, 256, (N // 16, K_ // 128, 1024), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.full((N // 16, K_ // 128, 64), 127, device="cuda", dtype=torch.uint8)
    a, sa = whole_codes(T, K_, g)
    out = qm.moe_gemm_mx(a, sa, "fp4", w, ws, N, out_dtype=torch.float32)
    for lo in (0, 2_100, N // 16 - 40):
        part = qm.moe_gemm_mx(a, sa, "fp4", w[lo:lo + 40].contiguous(), ws[lo:lo + 40].contiguous(), 640, out_dtype=torch.float32)
        assert torch.equal(out[:, 16 * lo:16 * lo + 640], part)


def test_tokens_past_2_32_bytes():
    g = torch.Generator(device="cuda").manual_seed(9)
    T, K_, N = 132_000, 65_536, 48
    a, sa = whole_codes(T, K_, g)
    w, ws = qm.moe_pack_mx(*whole_codes(N, K_, g))
    out = qm.moe_gemm_mx(a, sa, "fp4", w, ws, N, out_dtype=torch.float32)
    for lo in (0, 70_001, T - 200):
        part = qm.moe_gemm_mx(a[lo:lo + 200].contiguous(), sa[lo:lo + 200].contiguous(), "fp4", w, ws, N, out_dtype=torch.float32)
        assert torch.equal(out[lo:lo + 200], part)


def test_strided_or_mistyped_tensors_are_refused():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="strided"):
        qm.moe_layer_norm(x[:, ::2])
    with pytest.raises(ValueError, match="noise"):
        qm.moe_quant_mx(x, "fp8", noise=torch.zeros(4, 128, dtype=torch.uint8))
    with pytest.raises(ValueError, match="w"):
        qm.moe_layer_norm(x, w=torch.ones(128))
    with pytest.raises(qm.MoeError, match="UNSUPPORTED"):
        qm.moe_quant_mx(x, "fp8", packed=True)
    with pytest.raises(qm.MoeError, match="UNSUPPORTED"):
        qm.moe_layer_norm(torch.zeros(2, 20000, device="cuda"))
    with pytest.raises(ValueError, match="w:"):
        qm.moe_gemm_mx(x.view(torch.uint8)[:, :64].contiguous(), torch.zeros(4, 2, dtype=torch.uint8, device="cuda"), "fp8",
                       x.view(torch.uint8), x.view(torch.uint8), 16)
