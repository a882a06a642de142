"""One whole MoE layer through the library, as a program runs it: the norms around the blocks, the
router, the sort and the routed experts, the int8 shared expert, and the next norm; each step
against float64 on the inputs the GPU gave it, and the chain end to end.  Also captured in HIP graphs,
replayed with new inputs, with two graphs alive, and on another stream, every time with the bits of
the eager run."""
import numpy as np
import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm
from oracle import moe as om
from quantized_moe_expert_sort_amd import inputs as gen

pytestmark = pytest.mark.gpu
D, E, K, I, SHARED = 256, 16, 4, 128, 192
EPS = 1e-6
SITU = dict(beta=gen.BETA, linear_beta=gen.LINEAR_BETA)


@pytest.fixture(scope="module")
def weights():
    g = torch.Generator().manual_seed(21)
    n = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int32).to(torch.int8)   # noqa: E731
    host = {"post": 1 + 0.2 * n(D), "pre": 1 + 0.2 * n(D), "post2": 1 + 0.2 * n(D), "pre2": 1 + 0.2 * n(D),
            "router": n(E, D) / D ** 0.5, "bias": 0.05 * n(E),
            "s1": codes(2 * SHARED, D), "c1": torch.rand(2 * SHARED, generator=g) / (40 * D ** 0.5),
            "s2": codes(D, SHARED), "c2": torch.rand(D, generator=g) / (40 * SHARED ** 0.5)}
    dev = {k: v.cuda() for k, v in host.items()}
    dev["s1"], dev["s2"] = qm.moe_pack_i8(dev["s1"]), qm.moe_pack_i8(dev["s2"])
    experts = gen.make_weights(7, E, D, I)
    return host, dev, experts, qm.device_weights(*experts)


def inputs(T, seed=0):
    g = torch.Generator().manual_seed(100 * seed + T)
    return {"x": (2 * torch.randn(T, D, generator=g)).bfloat16().cuda(), "y": torch.randn(T, D, generator=g).bfloat16().cuda(),
            "gate": torch.randn(T, generator=g).cuda()}


def layer(w, experts, s):
    """Every intermediate of one layer, in the order of the calls."""
    T = s["x"].shape[0]
    o = {}
    a = qm.moe_block_norm(s["x"], s["y"], w_post=w["post"], w_pre=w["pre"], eps=EPS, q_dtype="i8")
    o.update(h=a.h, n=a.n, q=a.q, qs=a.q_scale)
    o["logits"] = a.n.float() @ w["router"].t()
    r = qm.moe_router(o["logits"], K, score="sigmoid", bias=w["bias"], scale=1.5)
    o.update(ids=r.ids, w=r.w)
    lay = qm.moe_sort(r.ids, r.w, 0, E, qm.block_m(T))
    o["routed"] = qm.moe_fused(a.n, None, "bf16", *experts, r.w, lay, E, "situv2", gen.BETA, gen.LINEAR_BETA)
    o["mid"] = qm.moe_gemm_i8(a.q, a.q_scale, w["s1"], w["c1"], act="situv2", **SITU)
    o["mq"], o["ms"] = qm.moe_quant_i8(o["mid"])
    o["out"] = qm.moe_gemm_i8(o["mq"], o["ms"], w["s2"], w["c2"], add=o["routed"])
    b = qm.moe_block_norm(a.h, o["out"], w_post=w["post2"], gate=s["gate"], gate_kind="token", gate_act="sigmoid",
                          scale=0.5, w_pre=w["pre2"], eps=EPS, q_dtype="fp8")
    o.update(h2=b.h, n2=b.n, q2=b.q, q2s=b.q_scale)
    return o


def rel(got, want):
    return float((ref.f64(got) - want).norm() / want.norm())


@pytest.mark.parametrize("T", [1, 37, 300])
def test_layer_against_float64(T, weights):
    host, dev, experts, experts_dev = weights
    s = inputs(T)
    o = layer(dev, experts_dev, s)
    f = {k: ref.f64(v) for k, v in host.items()}
    x = {k: ref.f64(v) for k, v in s.items()}
    # step by step, on the GPU's own intermediates
    h, n, _ = ref.norm_forward(x["x"], x["y"], f["post"], None, "none", "none", 1.0, f["pre"], EPS)
    assert rel(o["h"], h) < ref.HALF_BF16 and rel(o["n"], n) < ref.HALF_BF16
    ids = ref.router_choice(o["logits"], K, "sigmoid", host["bias"])
    assert torch.equal(o["ids"].cpu(), ids)
    lm = ref.masked_logits(o["logits"])
    w, _, _, _ = ref.router_outputs(lm, ids, "sigmoid", True, 1.5, torch.ones(T, dtype=torch.bool), 0.0, 0.0)
    assert rel(o["w"], w) < 1e-5
    bits = o["n"].view(torch.int16).cpu().numpy().view(np.uint16)
    routed = torch.from_numpy(om.moe_fused(bits, "bf16", *experts, ids.numpy(), o["w"].cpu().numpy(), 0, E, "situv2",
                                           gen.BETA, gen.LINEAR_BETA))
    assert rel(o["routed"], routed) < 5e-3
    mid, err = ref.gemm_i8(o["q"], o["qs"], host["s1"], host["c1"], "situv2")
    assert ((ref.f64(o["mid"]) - mid).abs() <= ref.HALF_BF16 * mid.abs() + 1.01 * err).all()
    wq, ws = ref.quant_i8(o["mid"].cpu())
    assert torch.equal(o["mq"].cpu(), wq) and torch.equal(o["ms"].cpu(), ws)
    out, err = ref.gemm_i8(o["mq"], o["ms"], host["s2"], host["c2"], add=o["routed"])
    assert ((ref.f64(o["out"]) - out).abs() <= ref.HALF_BF16 * out.abs() + 1.01 * err).all()
    h2, n2, _ = ref.norm_forward(ref.f64(o["h"]), ref.f64(o["out"]), f["post2"], x["gate"], "token", "sigmoid", 0.5,
                                 f["pre2"], EPS)
    assert rel(o["h2"], h2) < ref.HALF_BF16 and rel(o["n2"], n2) < ref.HALF_BF16
    # end to end in float64, with the GPU's choice of experts: an int8 code is off by up to half of
    # amax / 127, about 0.8% of a row's rms, twice in a row, on the shared part alone; the routed
    # part carries bf16 roundings and the residual stream neither
    g, u = ((n @ (f["s1"] * f["c1"][:, None]).t())).chunk(2, 1)
    m = gen.BETA * torch.tanh(g / gen.BETA) * torch.sigmoid(g) * gen.LINEAR_BETA * torch.tanh(u / gen.LINEAR_BETA)
    shared = m @ (f["s2"] * f["c2"][:, None]).t()
    assert rel(o["out"] - o["routed"], shared) < 3e-2 + ref.HALF_BF16 * 2 * float(routed.norm() / shared.norm())
    hh, nn, _ = ref.norm_forward(h, shared + routed, f["post2"], x["gate"], "token", "sigmoid", 0.5, f["pre2"], EPS)
    assert rel(o["h2"], hh) < 3e-2 and rel(o["n2"], nn) < 3e-2


def equal(a, b):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8) if a[k].dtype == torch.float8_e4m3fn else a[k], b[k]), k


def captured(fn, s):
    for _ in range(2):                                          # sizes and workspaces settle before the capture
        fn(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn(s)
    return graph, out


def test_layer_in_graphs(weights):
    _, dev, _, experts = weights
    small, large = inputs(5), inputs(200)
    run = lambda s: layer(dev, experts, s)   # noqa: E731
    graphs = [(s, *captured(run, s)) for s in (small, large)]  # both alive at once
    for turn in range(4):
        for s, graph, out in graphs:
            new = inputs(s["x"].shape[0], seed=turn + 1)
            want = {k: v.clone() for k, v in run(new).items()}
            for k in s:
                s[k].copy_(new[k])
            graph.replay()
            torch.cuda.synchronize()
            equal(want, out)


def train(s):
    """Norm pair and router with losses, forward and backward."""
    kw = dict(w_post=s["wo"], gate=s["g"], gate_kind="channel", gate_act="sigmoid", w_pre=s["wi"])
    r = qm.moe_block_norm(s["x"], s["y"], stats=True, **kw)
    t = qm.moe_router(s["logits"], 6, score="sigmoid", bias=s["bias"], balance=(0.1, 0.01), valid=s["valid"])
    dl = qm.moe_router_backward(s["logits"], t, s["dw"], d_loss=s["dloss"], score="sigmoid", valid=s["valid"])
    b = qm.moe_block_norm_backward(s["x"], s["y"], r.rstd, s["dh"], s["dn"], **kw)
    return dict(h=r.h, n=r.n, ids=t.ids, w=t.w, counts=t.balance.counts, mean=t.balance.mean_prob, loss=t.balance.loss,
                dl=dl, **b._asdict())


def train_inputs(T, seed=0):
    g = torch.Generator().manual_seed(300 * seed + T)
    n = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    return {"x": n(T, 520), "y": n(T, 520).bfloat16(), "wo": n(520), "wi": n(520), "g": n(520), "dh": n(T, 520),
            "dn": n(T, 520).bfloat16(), "logits": n(T, 100), "bias": 0.1 * n(100), "dw": n(T, 6), "dloss": n(2),
            "valid": (torch.rand(T, generator=g) < 0.8).cuda()}


def test_training_step_in_graphs():
    first, second = train_inputs(70), train_inputs(600)
    graphs = [(s, *captured(train, s)) for s in (first, second)]
    for turn in range(4):
        for s, graph, out in graphs:
            new = train_inputs(s["x"].shape[0], seed=turn + 1)
            want = {k: v.clone() for k, v in train(new).items()}
            for k in s:
                s[k].copy_(new[k])
            graph.replay()
            torch.cuda.synchronize()
            equal(want, out)


def test_on_another_stream(weights):
    _, dev, _, experts = weights
    s, t = inputs(64), train_inputs(90)
    want, want_t = layer(dev, experts, s), train(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, got_t = layer(dev, experts, s), train(t)
    side.synchronize()
    equal(want, got)
    equal(want_t, got_t)


def test_two_streams_at_once():
    # each call has a workspace of its own: runs that overlap in time do not touch each other
    cases = [train_inputs(2000, seed=i) for i in range(2)]
    want = [{k: v.clone() for k, v in train(c).items()} for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (c, st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                got[i] = train(c)
    torch.cuda.synchronize()
    for i in range(2):
        equal(want[i], got[i])


def test_strided_or_mistyped_tensors_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="strided"):
        qm.moe_block_norm(x[:, ::2], w_pre=w[:32])
    with pytest.raises(ValueError, match="w_pre"):
        qm.moe_block_norm(x, w_pre=w.bfloat16())
    with pytest.raises(ValueError, match="y"):
        qm.moe_block_norm(x, x[:2], w_post=w)
    with pytest.raises(ValueError, match="bias"):
        qm.moe_router(x, 2, bias=w.cpu())
    with pytest.raises(qm.MoeError, match="UNSUPPORTED"):
        qm.moe_router(x, 40)
    with pytest.raises(qm.MoeError, match="INVALID"):
        qm.moe_router(x, 0)
    with pytest.raises(ValueError, match="w_packed"):
        qm.moe_gemm_i8(x.to(torch.int8), w[:4], x.to(torch.int8), w)
    with pytest.raises(qm.MoeError, match="UNSUPPORTED"):
        qm.moe_block_norm(torch.zeros(2, 40, dtype=torch.bfloat16, device="cuda"), w_pre=w[:40].clone(), q_dtype="fp8")
