"""The operators around the routed experts on more rows than one dispatch holds work items for (2^32
in a dimension, 64 or more a row): every row has to give what it gives in a short batch."""
import pytest
import torch

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


def rows(b):
    """The block over and over, T rows."""
    out = torch.empty(T, *b.shape[1:], dtype=b.dtype, device="cuda")
    out[:T // BLOCK * BLOCK].view(-1, *b.shape).copy_(b.expand(T // BLOCK, *b.shape))
    out[T // BLOCK * BLOCK:] = b[:T % BLOCK]
    return out


def same(big, b, what):
    whole = big[:T // BLOCK * BLOCK].view(-1, *b.shape)
    for part in whole.split(512):
        assert (part == b).all(), what
    assert torch.equal(big[T // BLOCK * BLOCK:], b[:T % BLOCK]), what


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


@pytest.mark.parametrize("gate_kind,q_dtype,D", [("token", "i8", 16), ("element", "fp8", 32), ("channel", None, 7)])
def test_block_norm(gate_kind, q_dtype, D):
    x, y = block(D), block(D, seed=1)
    gate = {"token": lambda: block(seed=2, dtype=torch.float32), "element": lambda: block(D, seed=2),
            "channel": lambda: torch.rand(D, device="cuda")}[gate_kind]()
    kw = dict(w_post=torch.rand(D, device="cuda") + 0.5, w_pre=torch.rand(D, device="cuda") + 0.5, gate_kind=gate_kind,
              gate_act="sigmoid", q_dtype=q_dtype, stats=True)
    small = qm.moe_block_norm(x, y, gate=gate, **kw)
    big = qm.moe_block_norm(rows(x), rows(y), gate=gate if gate_kind == "channel" else rows(gate), **kw)
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
