"""The operators around the routed experts on more rows than one dispatch holds work items for (2^32
in a dimension, 64 or more a row): every row has to give what it gives in a short batch."""
import pytest
import torch

import _layer_ref as ref
import quantized_moe_expert_sort_amd as qm

pytestmark = pytest.mark.gpu
BLOCK = 1 << 14                                                # random rows, repeated
T = (1 << 26) + 5                                              # 64 work items a row: just over 2^32


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def block(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(BLOCK, *shape, device="cuda", generator=g).to(dtype)


def rows(b, T=T):
    """The block over and over, T rows."""
    out = torch.empty(T, *b.shape[1:], dtype=b.dtype, device="cuda")
    n = b.shape[0]
    out[:T // n * n].view(-1, *b.shape).copy_(b.expand(T // n, *b.shape))
    out[T // n * n:] = b[:T % n]
    return out


def same(big, b, what):
    n = b.shape[0]
    whole = big[:big.shape[0] // n * n].view(-1, *b.shape)
    for part in whole.split(512):
        assert (part == b).all(), what
    assert torch.equal(big[whole.shape[0] * n:], b[:big.shape[0] % n]), what


def test_router():
    b = block(8)
    valid = torch.rand(BLOCK, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.8
    small = qm.moe_router(b, 2, valid=valid)
    logits = rows(b)
    big = qm.moe_router(logits, 2, valid=rows(valid))
    same(big.ids, small.ids, "ids")
    same(big.w, small.w, "w")
    biased = qm.moe_router(logits, 3, score="sigmoid", bias=torch.arange(8, device="cuda") / 8.0)
    same(biased.ids, qm.moe_router(b, 3, score="sigmoid", bias=torch.arange(8, device="cuda") / 8.0).ids, "ids with a bias")


@pytest.mark.parametrize("gate_kind,q_dtype,D", [("token", "i8", 16), ("element", "fp8", 32), ("none", "fp4", 32),
                                                   ("channel", None, 7)])
def test_block_norm(gate_kind, q_dtype, D):
    x, y = block(D), block(D, seed=1)
    gate = {"token": lambda: block(seed=2, dtype=torch.float32), "element": lambda: block(D, seed=2),
            "channel": lambda: torch.rand(D, device="cuda"), "none": lambda: None}[gate_kind]()
    kw = dict(w_post=torch.rand(D, device="cuda") + 0.5, w_pre=torch.rand(D, device="cuda") + 0.5, gate_kind=gate_kind,
              gate_act="none" if gate is None else "sigmoid", q_dtype=q_dtype, stats=True)
    small = qm.moe_block_norm(x, y, gate=gate, **kw)
    big = qm.moe_block_norm(rows(x), rows(y), gate=gate if gate_kind in ("channel", "none") else rows(gate), **kw)
    for k in ("h", "n") + (("q", "q_scale") if q_dtype else ()):
        same(getattr(big, k), getattr(small, k), k)
    same(big.rstd[0], small.rstd[0], "1/rms(y)")
    same(big.rstd[1], small.rstd[1], "1/rms(h)")


def test_quant():
    b = block(16)
    q, s = qm.moe_quant_i8(rows(b))
    ql, sl = qm.moe_quant_i8(b)
    same(q, ql, "codes")
    same(s, sl, "scales")


def test_block_norm_of_as_many_rows_as_an_int_counts():
    # rows of one element: 1/rms is 1 (eps is below the last place), so dx = dh, and dw_pre counts the rows
    n = (1 << 31) - 1
    x = torch.ones(n, 1, dtype=torch.bfloat16, device="cuda")
    w = torch.full((1,), 2.0, device="cuda")
    r = qm.moe_block_norm(x, w_pre=w, eps=1e-12, stats=True)
    assert all((part == 2).all() for part in r.n.split(1 << 28))
    b = qm.moe_block_norm_backward(x, None, r.rstd, x, x, w_pre=w)
    assert all((part == 1).all() for part in b.dx.split(1 << 28))
    assert float(b.dw_pre) == 2.0 ** 31                        # rounded to fp32


@pytest.mark.parametrize("gate_kind", ["token", "element", "none"])
@pytest.mark.parametrize("n,D,x_dt", [((1 << 20) + 256, 8, torch.bfloat16), (40_192, 8200, torch.float32)])
def test_backward_in_slices(n, D, x_dt, gate_kind):
    # rows enough for the sums over them to be taken in more than one launch
    b = 256
    g = torch.Generator(device="cuda").manual_seed(3)
    make = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
    one = {"x": make(b, D).to(x_dt), "y": make(b, D).to(torch.bfloat16), "dh": make(b, D).to(x_dt), "dn": make(b, D).to(torch.bfloat16)}
    gate = {"token": lambda: make(b), "element": lambda: make(b, D).to(torch.bfloat16), "none": lambda: None}[gate_kind]()
    kw = dict(w_post=make(D), w_pre=make(D), gate_kind=gate_kind, gate_act="none" if gate is None else "sigmoid")
    r = qm.moe_block_norm(one["x"], one["y"], gate=gate, stats=True, **kw)
    want = qm.moe_block_norm_backward(one["x"], one["y"], r.rstd, one["dh"], one["dn"], gate=gate, **kw)
    many = {k: rows(v, n) for k, v in one.items()}
    rstd = torch.stack((rows(r.rstd[0].contiguous(), n), rows(r.rstd[1].contiguous(), n)))
    got = qm.moe_block_norm_backward(many["x"], many["y"], rstd, many["dh"], many["dn"], dx=many["dh"],
                                     gate=None if gate is None else rows(gate, n), **kw)
    for k in ("dx", "dy", "dgate"):
        if getattr(want, k) is not None:
            same(getattr(got, k), getattr(want, k), k)
    # the sums: as many times the block's, within the bounds of the norm's tests
    f = ref.f64
    exact, m = ref.norm_backward(f(one["x"]), f(one["y"]), f(kw["w_post"]), f(gate), gate_kind, kw["gate_act"], 1.0, f(kw["w_pre"]), 1e-6,
                                 f(one["dh"]), f(one["dn"]))
    for k in ("dw_post", "dw_pre"):
        off = (f(getattr(got, k)) - n // b * exact[k]).abs()
        assert (off <= n // b * (3 * 64 * ref.HALF_F32 * m[k] + ref.HALF_F32 * exact[k].abs())).all(), k
