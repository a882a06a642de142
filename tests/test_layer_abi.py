"""The operators around the routed experts refuse bad arguments on the host, through the C ABI (with
placeholder pointers, so only where no GPU is visible) and through the Python binding, and the
binding's structs and size helpers match the header."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import quantized_moe_expert_sort_amd as qm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_mi355x.h")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: CPU-only checks")

P = 0x100000                           # placeholder device pointer (never dereferenced)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
NAN, INF = float("nan"), float("inf")


def struct_fields(name):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^{}]*)\} " + name + ";", src).group(1)
    out = []
    for decl in body.split(";"):
        m = re.match(r"\s*(?:const )?(\w+)\s+(.*)", decl.strip(), flags=re.S)
        if m:
            for field in m.group(2).split(","):
                ptr = "*" in field
                out.append((field.replace("*", "").strip(), "ptr" if ptr else m.group(1)))
    return out


@pytest.mark.parametrize("name,py", [("moe_block_norm_t", qm.BlockNormParams), ("moe_block_norm_grads_t", qm.BlockNormGradParams),
                                     ("moe_router_t", qm.RouterParams), ("moe_balance_t", qm.BalanceParams)])
def test_structs_match_the_header(name, py):
    kinds = {ctypes.c_void_p: "ptr", ctypes.c_int32: "int32_t", ctypes.c_float: "float"}
    assert struct_fields(name) == [(n, kinds[t]) for n, t in py._fields_]


def test_size_helpers_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    norm = [(0, 64), (1, 3584), (5, 1790), (511, 16384), (512, 8), (9999, 3584)]
    i8 = [(1, 16), (7168, 3584), (1000, 1456), (17, 144)]
    lines = ['printf("%%zu\\n", moe_block_norm_backward_ws_bytes(%d, %d));' % c for c in norm]
    lines += ['printf("%%zu\\n", moe_router_ws_bytes(%d));' % e for e in (1, 896, 2048)]
    lines += ['printf("%%zu\\n", moe_i8_packed_bytes(%d, %d));' % c for c in i8]
    lines += ['printf("%d %d %d %d\\n", MOE_NORM_MAX_DIM, MOE_NORM_PARTS, MOE_ROUTER_MAX_TOPK, MOE_ROUTER_PARTS);']
    src.write_text('#include <stdio.h>\n#include "moe_mi355x.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-O1", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = [qm.block_norm_backward_ws_bytes(*c) for c in norm] + [qm.router_ws_bytes(e) for e in (1, 896, 2048)]
    for n, k in i8:
        a, b, c = qm.i8_packed_shape(n, k)
        want.append(a * b * c)
    want += [qm.NORM_MAX_DIM, qm.NORM_PARTS, qm.ROUTER_MAX_TOPK, qm.ROUTER_PARTS]
    assert [int(v) for v in got] == want


def norm(**kw):
    f = dict(x=P, y=P, w_post=P, gate=None, w_pre=P, h=P, n=P, q=None, q_scale=None, rstd=None, tokens=4, dim=64, x_dt=0,
             gate_kind=0, gate_act=0, q_dt=0, scale=1.0, eps=1e-6)
    f.update(kw)
    return qm.BlockNormParams(**f)


def norm_status(**kw):
    return qm.lib().moe_block_norm(norm(**kw), None)


@no_gpu
def test_block_norm_refusals():
    assert qm.lib().moe_block_norm(None, None) == INVALID
    for bad in (dict(tokens=-1), dict(dim=0), dict(dim=-5), dict(x_dt=1), dict(x_dt=4), dict(gate_kind=4), dict(gate_kind=-1),
                dict(gate_act=2), dict(gate_act=1), dict(scale=NAN), dict(scale=INF), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=1e-40),
                dict(gate=P), dict(gate_kind=1), dict(x=None), dict(y=None), dict(y=None, w_post=None, gate=P, gate_kind=2),
                dict(w_pre=None), dict(h=None, n=None), dict(q=P), dict(q_scale=P), dict(q=P, q_scale=P, q_dt=0),
                dict(q=P, q_scale=P, q_dt=3), dict(q=P, q_scale=P, q_dt=1, n=None, w_pre=None),
                dict(q=P, q_scale=P, q_dt=1, x=P + 2), dict(q=P + 8, q_scale=P, q_dt=4), dict(q=P, q_scale=P, q_dt=2, n=P + 8),
                dict(q=P, q_scale=P, q_dt=2, gate=P + 4, gate_kind=1)):
        assert norm_status(**bad) == INVALID, bad
    assert norm_status(dim=16385) == UNSUPPORTED
    assert norm_status(dim=48, q=P, q_scale=P, q_dt=1) == UNSUPPORTED
    assert norm_status(dim=40, q=P, q_scale=P, q_dt=4) == UNSUPPORTED
    assert norm_status(tokens=0, x=None) == OK


def backward_status(ws=P, ws_bytes=1 << 30, grads=None, **kw):
    g = dict(dh=P, dn=P, dx=P, dy=P, dgate=None, dw_post=P, dw_pre=P)
    g.update(grads or {})
    kw.setdefault("rstd", P)
    return qm.lib().moe_block_norm_backward(norm(**kw), qm.BlockNormGradParams(**g), ws, ws_bytes, None)


@no_gpu
def test_block_norm_backward_refusals():
    assert qm.lib().moe_block_norm_backward(norm(rstd=P), None, P, 1 << 30, None) == INVALID
    for g in (dict(dh=None, dn=None, dw_pre=None), dict(dx=None), dict(dy=None), dict(dgate=P), dict(dw_post=None),
              dict(dw_pre=None), dict(dn=None)):
        assert backward_status(grads=g) == INVALID, g
    assert backward_status(w_pre=None) == INVALID
    assert backward_status(rstd=None) == INVALID
    assert backward_status(gate=P, gate_kind=1) == INVALID              # no dgate
    assert backward_status(ws=None) == INVALID
    assert backward_status(ws_bytes=qm.block_norm_backward_ws_bytes(4, 64) - 1) == WORKSPACE
    assert backward_status(dim=20000) == UNSUPPORTED


def router(**kw):
    f = dict(logits=P, bias=None, valid=None, topk_ids=P, topk_w=P, tokens=4, num_experts=8, topk=2, dt=0, score=0, renorm=1,
             scale=1.0)
    f.update(kw)
    return qm.RouterParams(**f)


BAL = dict(coef=1.0, z_coef=0.0, counts=P, mean_prob=P, loss=P, num_valid=P)


@no_gpu
def test_router_refusals():
    f, b = qm.lib().moe_router, qm.lib().moe_router_backward
    bal = lambda **kw: qm.BalanceParams(**dict(BAL, **kw))   # noqa: E731
    assert f(None, None, None, 0, None) == INVALID and b(None, None, P, None, P, None) == INVALID
    for bad in (dict(tokens=-1), dict(num_experts=0), dict(topk=0), dict(dt=1), dict(dt=4), dict(score=2), dict(renorm=2),
                dict(scale=INF), dict(logits=None), dict(topk_ids=None)):
        assert f(router(**bad), None, None, 0, None) == INVALID, bad
        assert b(router(**bad), None, P, None, P, None) == INVALID, bad
    assert f(router(topk_w=None), None, None, 0, None) == INVALID
    for bad in (dict(num_experts=2049), dict(topk=9), dict(topk=33, num_experts=64), dict(tokens=(1 << 31) - 1, num_experts=2048)):
        assert f(router(**bad), None, None, 0, None) == UNSUPPORTED, bad
        assert b(router(**bad), None, P, None, P, None) == UNSUPPORTED, bad
    need = qm.router_ws_bytes(8)
    for bad in (dict(coef=NAN), dict(z_coef=INF), dict(counts=None), dict(mean_prob=None), dict(loss=None), dict(num_valid=None)):
        assert f(router(), bal(**bad), P, need, None) == INVALID, bad
    assert f(router(), bal(), None, need, None) == INVALID
    assert f(router(), bal(), P, need - 1, None) == WORKSPACE
    assert f(router(tokens=0), None, None, 0, None) == OK
    assert b(router(), None, None, None, P, None) == INVALID            # nothing to differentiate
    assert b(router(), None, P, None, None, None) == INVALID
    assert b(router(), bal(counts=None), P, None, P, None) == INVALID
    assert b(router(), bal(num_valid=None), P, None, P, None) == INVALID
    assert b(router(tokens=0), None, None, None, None, None) == OK


@no_gpu
def test_int8_refusals():
    L = qm.lib()
    assert L.moe_quant_i8(P, 4, 24, P, P, None) == INVALID
    assert L.moe_quant_i8(P, -1, 32, P, P, None) == INVALID
    assert L.moe_quant_i8(P, 4, 0, P, P, None) == INVALID
    assert L.moe_quant_i8(P + 2, 4, 32, P, P, None) == INVALID
    assert L.moe_quant_i8(None, 4, 32, P, P, None) == INVALID
    assert L.moe_quant_i8(P, 1 << 31, 32, P, P, None) == UNSUPPORTED
    assert L.moe_quant_i8(None, 0, 32, None, None, None) == OK
    far = 0x40000000
    assert L.moe_pack_i8(None, 16, 64, far, None) == INVALID
    assert L.moe_pack_i8(P, 0, 64, far, None) == INVALID
    assert L.moe_pack_i8(P, 16, 64, P, None) == INVALID
    assert L.moe_pack_i8(P, 16, 64, P + 1008, None) == INVALID
    assert L.moe_pack_i8(P + 2032, 16, 64, P, None) == INVALID          # the packed rows are padded to 128 bytes
    assert L.moe_pack_i8(P + 8, 16, 64, far, None) == INVALID
    assert L.moe_pack_i8(P, 16, 72, far, None) == UNSUPPORTED
    assert L.moe_pack_i8(P, 1 << 22, 1 << 10, 1 << 40, None) == UNSUPPORTED

    def gemm(a=P, sa=P, w=P, sw=P, T=4, N=64, K=64, act=None, add=None, out=P):
        return L.moe_gemm_i8(a, sa, w, sw, T, N, K, act, add, out, None)
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None),
                dict(a=P + 8), dict(w=P + 4), dict(act=qm.ActParams(0, 0.0, 25.0)), dict(act=qm.ActParams(0, 4.0, NAN))):
        assert gemm(**bad) == INVALID, bad
    for bad in (dict(K=72), dict(K=1 << 17), dict(N=48, act=qm.ActParams(1, 0.0, 0.0)), dict(act=qm.ActParams(2, 1.0, 1.0)),
                dict(T=1 << 24), dict(N=1 << 30, K=64)):
        assert gemm(**bad) == UNSUPPORTED, bad
    assert gemm(T=0, a=None) == OK


def test_binding_refuses_tensors_off_the_gpu_and_unknown_names():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: qm.moe_block_norm(x), lambda: qm.moe_block_norm_backward(x, None, None, x, None),
                 lambda: qm.moe_router(x, 2), lambda: qm.moe_router_backward(x, None), lambda: qm.moe_quant_i8(x),
                 lambda: qm.moe_pack_i8(x), lambda: qm.moe_gemm_i8(x, None, None, None)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    dev = -1                                                   # the index of a tensor on the CPU
    with pytest.raises(ValueError, match="gate_kind"):
        qm._norm_params(x, None, None, None, "row", "none", 1.0, None, 1e-6, dev)
    with pytest.raises(ValueError, match="go together"):
        qm._norm_params(x, x, None, None, "token", "none", 1.0, None, 1e-6, dev)
    with pytest.raises(ValueError, match="w_pre"):
        qm._norm_params(x, x, None, None, "none", "none", 1.0, torch.ones(64, dtype=torch.bfloat16), 1e-6, dev)
    with pytest.raises(ValueError, match="strided"):
        qm._norm_params(x, torch.zeros(64, 2, dtype=torch.bfloat16).t(), None, None, "none", "none", 1.0, None, 1e-6, dev)
    with pytest.raises(ValueError, match="score"):
        qm._router_params(x, 2, "relu", True, 1.0, None, None, dev)
    with pytest.raises(ValueError, match="bias"):
        qm._router_params(x, 2, "sigmoid", True, 1.0, torch.zeros(63), None, dev)
    with pytest.raises(ValueError, match="logits"):
        qm._router_params(x.half(), 2, "sigmoid", True, 1.0, None, None, dev)


@no_gpu
def test_workspaces_have_to_be_aligned_like_their_words():
    # the workspaces hold 4-byte words, among them one that is counted up by atomics
    need = qm.router_ws_bytes(8)
    for off in (1, 2, 3):
        assert qm.lib().moe_router(router(), qm.BalanceParams(**BAL), P + off, need, None) == INVALID, off
        assert qm.lib().moe_router(router(tokens=0), qm.BalanceParams(**BAL), P + off, need, None) == INVALID, off
        assert backward_status(ws=P + off) == INVALID, off
        # where no workspace is read, its address does not matter
        assert qm.lib().moe_router(router(tokens=0), None, P + off, 0, None) == OK, off


def test_binding_refuses_sizes_that_its_32_bit_fields_would_wrap(monkeypatch):
    # 2^32 + 5 rows would arrive as 5; tensors without storage stand for ones of that size
    def reached(fn, *args):
        raise AssertionError(f"{fn} was called")
    monkeypatch.setattr(qm, "_on_gpu", lambda t, name: (t.device, t.get_device()))
    monkeypatch.setattr(qm, "_call", reached)
    big = (1 << 32) + 16

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")
    i8, f32, i32 = torch.int8, torch.float32, torch.int32
    w = empty(1, dtype=f32)
    ids = empty(big, 1, dtype=i32)
    packed = empty(*qm.i8_packed_shape(16, 16), dtype=i8)
    for call in (lambda: qm.moe_block_norm(empty(big, 1), w_pre=w, want_n=False, h=empty(big, 1)),
                 lambda: qm.moe_block_norm(empty(1, big), h=empty(1, big)),
                 lambda: qm.moe_block_norm_backward(empty(big, 1), None, empty(2, big, dtype=f32), None, empty(big, 1), w_pre=w),
                 lambda: qm.moe_router(empty(big, 1), 1),
                 lambda: qm.moe_router(empty(1, big), 1),
                 lambda: qm.moe_router(empty(0, 8), big),
                 lambda: qm.moe_router(empty(1, 8), 2 - (1 << 32)),
                 lambda: qm.moe_router_backward(empty(big, 1), qm.Routing(ids, None, None), empty(big, 1, dtype=f32)),
                 lambda: qm.moe_pack_i8(empty(big, 16, dtype=i8)),
                 lambda: qm.moe_pack_i8(empty(16, big, dtype=i8)),
                 lambda: qm.moe_gemm_i8(empty(big, 16, dtype=i8), empty(big, dtype=f32), packed, empty(16, dtype=f32)),
                 lambda: qm.moe_gemm_i8(empty(1, big, dtype=i8), empty(1, dtype=f32), packed, empty(16, dtype=f32)),
                 lambda: qm.moe_gemm_i8(empty(1, 16, dtype=i8), empty(1, dtype=f32), packed, empty(big, dtype=f32))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_import_needs_nothing_of_torch_beyond_its_public_names():
    # a build of torch without the private getters of device and stream: the package imports, and calls
    # take both from torch.cuda
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import quantized_moe_expert_sort_amd as qm
class Stream:
    cuda_stream = 77
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda index: Stream
assert qm._current_device() == 3 and qm._raw_stream(3) == 77
assert not torch.cuda.is_initialized()
print("imported")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
