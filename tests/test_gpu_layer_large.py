"""The operators around the routed experts on tensors of more than 2^31 elements: the last rows have
to give the bits that the same rows give alone, and the sums over rows those of the rows that are
not zero."""
import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
ROWS = 3                                                       # random rows at the end


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def tail(T, D, dtype, seed):
    """(zeros [T, D] with random last rows, those rows alone)"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    last = torch.randn(ROWS, D, device="cuda", generator=g).to(dtype)
    full = torch.zeros(T, D, dtype=dtype, device="cuda")
    full[-ROWS:] = last
    return full, last


def test_block_norm():
    T, D = 140_000, 15_360                                     # 2.15e9 elements
    (x, xs), (y, ys), (dh, dhs), (dn, dns) = (tail(T, D, torch.bfloat16, s) for s in range(4))
    w, v = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    kw = dict(w_post=w, w_pre=v)
    big, small = (qm.moe_block_norm(a, b, stats=True, q_dtype="fp8", **kw) for a, b in ((x, y), (xs, ys)))
    for k in ("h", "n", "q", "q_scale"):
        assert torch.equal(getattr(big, k)[-ROWS:], getattr(small, k)), k
    assert torch.equal(big.rstd[:, -ROWS:], small.rstd)
    assert not big.h[:-ROWS].any() and not big.n[:-ROWS].any()
    rstd, srstd, n = big.rstd, small.rstd, small.n
    del big, small
    a = qm.moe_block_norm_backward(x, y, rstd, dh, dn, **kw)
    b = qm.moe_block_norm_backward(xs, ys, srstd, dhs, dns, **kw)
    assert torch.equal(a.dx[-ROWS:], b.dx) and torch.equal(a.dy[-ROWS:], b.dy)
    # zero rows add nothing; the sums of three terms may be added in another order: two roundings a
    # side of at most the sum of the terms' magnitudes (taken from bf16 outputs, so 1% more)
    terms = {"dw_pre": dns.float() * n.float() / v, "dw_post": b.dx.float() * ys.float() * srstd[0][:, None]}
    for k, t in terms.items():
        assert ((getattr(a, k) - getattr(b, k)).abs() <= 4 * 2.0 ** -24 * 1.01 * t.abs().sum(0)).all(), k


def test_router():
    T, E, K = 2_100_000, 1032, 2                               # 2.17e9 logits
    logits, last = tail(T, E, torch.bfloat16, 5)
    big, small = qm.moe_router(logits, K, balance=(0.1, 0.1)), qm.moe_router(last, K)
    assert torch.equal(big.ids[-ROWS:], small.ids) and torch.equal(big.w[-ROWS:], small.w)
    assert (big.ids[:-ROWS] == torch.tensor([0, 1], dtype=torch.int32, device="cuda")).all()
    assert int(big.balance.num_valid) == T and int(big.balance.counts.sum()) == T * K
    dw = torch.randn(T, K, device="cuda")
    a = qm.moe_router_backward(logits, big._replace(balance=None), dw)
    b = qm.moe_router_backward(last, small, dw[-ROWS:].clone())
    assert torch.equal(a[-ROWS:], b)


@pytest.mark.parametrize("T,N,K", [(2_000_000, 1100, 16), (1_050_000, 16, 4112)])
def test_product(T, N, K):                                     # 2.2e9 outputs; 4.3e9 bytes of tokens
    g = torch.Generator(device="cuda").manual_seed(9)
    last = torch.randint(-127, 128, (ROWS, K), device="cuda", generator=g, dtype=torch.int32).to(torch.int8)
    a = torch.zeros(T, K, dtype=torch.int8, device="cuda")
    a[-ROWS:] = last
    w = qm.moe_pack_i8(torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int32).to(torch.int8))
    sa, sw = torch.rand(T, device="cuda") + 0.5, torch.rand(N, device="cuda") / K
    out = qm.moe_gemm_i8(a, sa, w, sw)
    assert torch.equal(out[-ROWS:], qm.moe_gemm_i8(last, sa[-ROWS:].clone(), w, sw))
    assert not out[:-ROWS].any()


def test_quant():
    x, last = tail(140_000, 15_360, torch.bfloat16, 11)
    q, s = qm.moe_quant_i8(x)
    ql, sl = qm.moe_quant_i8(last)
    assert torch.equal(q[-ROWS:], ql) and torch.equal(s[-ROWS:], sl)
    assert not q[:-ROWS].any() and not s[:-ROWS].any()


@pytest.mark.parametrize("E,score,dt", [(7, "softmax", torch.bfloat16), (11, "sigmoid", torch.float32), (1030, "softmax", torch.bfloat16),
                                        (512, "softmax", torch.float32), (1024, "sigmoid", torch.bfloat16)])
def test_statistics_of_many_rows(E, score, dt):
    # rows that are all alike round alike: a chain of fp32 sums over all rows of a wave would be off by
    # up to the number of rows in it times 2^-24.  The bound is the same as for a short batch.
    T, K = min((1 << 24) + 77, (1 << 31) // E - 1), 3
    row = torch.linspace(-1.0, 1.0, E).to(dt)
    logits = row.cuda().expand(T, E).contiguous()
    r = qm.moe_router(logits, K, score=score, balance=(0.3, 0.02))
    l = row.double()
    p = torch.softmax(l if score == "softmax" else torch.nn.functional.logsigmoid(l), 0)
    rel = 128 * 2.0 ** -24                                     # as in the router's tests
    counts = torch.zeros(E, dtype=torch.int64)
    counts[ref.router_choice(row[None], K, score)[0].long()] = T
    assert torch.equal(r.balance.counts.cpu().long(), counts) and int(r.balance.num_valid) == T
    off = ((ref.f64(r.balance.mean_prob) - p).abs() / p).max()
    assert off <= 2 * rel, float(off / rel)
    want = torch.stack((0.3 * (counts * (E / (K * T)) * p).sum(), 0.02 * torch.logsumexp(l, 0).square()))
    off = ((ref.f64(r.balance.loss) - want).abs() / want).max()
    assert off <= 4 * rel, float(off / rel)


@pytest.mark.parametrize("T,D,dt", [((1 << 24) + 77, 8, torch.bfloat16), (2_000_003, 600, torch.float32), (300_007, 8200, torch.bfloat16)])
def test_weight_gradients_of_many_rows(T, D, dt):
    # as above: alike rows round alike, and the bound (that of the norm's tests) does not grow with them
    g = torch.Generator().manual_seed(D)
    x, dh = (torch.randn(1, D, generator=g).to(dt) for _ in range(2))
    y, dn = (torch.randn(1, D, generator=g).to(torch.bfloat16) for _ in range(2))
    w, v, gate = 1 + 0.3 * torch.randn(D, generator=g), 1 + 0.3 * torch.randn(D, generator=g), torch.randn(D, generator=g)
    kw = dict(w_post=w.cuda(), w_pre=v.cuda(), gate=gate.cuda(), gate_kind="channel", gate_act="sigmoid", scale=0.7)
    xs, ys, dhs, dns = (t.cuda().expand(T, D).contiguous() for t in (x, y, dh, dn))
    rstd = torch.empty(2, T, device="cuda")
    rstd.copy_(qm.moe_block_norm(x.cuda(), y.cuda(), eps=1e-5, stats=True, **kw).rstd.expand(2, T))
    b = qm.moe_block_norm_backward(xs, ys, rstd, dhs, dns, **kw)
    want, m = ref.norm_backward(*(t.double() for t in (x, y, w, gate)), "channel", "sigmoid", 0.7, v.double(), 1e-5, dh.double(), dn.double())
    for k in ("dw_post", "dw_pre", "dgate"):
        off = (ref.f64(getattr(b, k)) - T * want[k]).abs() / (T * (3 * 64 * 2.0 ** -24 * m[k] + 2.0 ** -24 * want[k].abs()))
        assert off.max() <= 1, (k, float(off.max()))
    for k in ("dx", "dy"):
        assert (getattr(b, k) == getattr(b, k)[:1]).all(), k
