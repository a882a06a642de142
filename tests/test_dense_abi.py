"""Layer norm and the microscaled matrices refuse bad arguments on the host, through the C ABI (with
placeholder pointers, so only where no GPU is visible) and through the Python binding, and the binding's
structs and size helpers match the header."""
import ctypes
import os
import subprocess

import pytest
import torch

import quantized_moe_expert_sort_amd as qm
from test_layer_abi import HEADER, INF, INVALID, NAN, OK, P, UNSUPPORTED, WORKSPACE, no_gpu, struct_fields


@pytest.mark.parametrize("name,py", [("moe_layer_norm_t", qm.LayerNormParams), ("moe_layer_norm_grads_t", qm.LayerNormGradParams),
                                     ("moe_quant_mx_t", qm.QuantMxParams)])
def test_structs_match_the_header(name, py):
    kinds = {ctypes.c_void_p: "ptr", ctypes.c_int32: "int32_t", ctypes.c_float: "float"}
    assert struct_fields(name) == [(n, kinds[t]) for n, t in py._fields_]


def test_size_helpers_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    norm = [(0, 64), (1, 3584), (5, 1790), (511, 16384), (9999, 3584)]
    mx = [(1, 1), (16, 128), (17, 129), (7168, 3584), (1000, 1790)]
    lines = ['printf("%%zu\\n", moe_layer_norm_backward_ws_bytes(%d, %d));' % c for c in norm]
    lines += ['printf("%%zu %%zu\\n", moe_mx_packed_bytes(%d, %d), moe_mx_packed_scale_bytes(%d, %d));' % (c + c) for c in mx]
    lines += ['printf("%d %d\\n", MOE_MX_ROWS, MOE_MX_PACKED);']
    src.write_text('#include <stdio.h>\n#include "moe_mi355x.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-O1", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = [qm.layer_norm_backward_ws_bytes(*c) for c in norm]
    for r, c in mx:
        for a, b, n in qm.mx_shapes(r, c, qm.DT_FP4, True):
            want.append(a * b * n)
    assert [int(v) for v in got] == want + [qm.MX_ROWS, qm.MX_PACKED]


def norm(**kw):
    f = dict(x=P, y=P, w=P, b=P, h=P, n=P, q=None, q_scale=None, stats=P, tokens=4, dim=64, x_dt=0, q_dt=0, eps=1e-5)
    f.update(kw)
    return qm.LayerNormParams(**f)


@no_gpu
def test_layer_norm_refusals():
    call = lambda **kw: qm.lib().moe_layer_norm(norm(**kw), None)   # noqa: E731
    assert qm.lib().moe_layer_norm(None, None) == INVALID
    for bad in (dict(tokens=-1), dict(dim=0), dict(x_dt=1), dict(x_dt=4), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
                dict(eps=1e-40), dict(x=None), dict(h=None, n=None, stats=None), dict(q=P), dict(q_scale=P),
                dict(q=P, q_scale=P, q_dt=0), dict(q=P, q_scale=P, q_dt=3), dict(q=P, q_scale=P, q_dt=1, x=P + 2),
                dict(q=P, q_scale=P, q_dt=1, b=P + 4), dict(q=P + 8, q_scale=P, q_dt=4)):
        assert call(**bad) == INVALID, bad
    assert call(dim=16385) == UNSUPPORTED
    assert call(dim=48, q=P, q_scale=P, q_dt=2) == UNSUPPORTED
    assert call(dim=40, q=P, q_scale=P, q_dt=4) == UNSUPPORTED
    assert call(tokens=0, x=None) == OK


@no_gpu
def test_layer_norm_backward_refusals():
    def call(ws=P, ws_bytes=1 << 30, grads=None, **kw):
        g = dict(dh=P, dn=P, dx=P, dy=P, dw=P, db=P)
        g.update(grads or {})
        return qm.lib().moe_layer_norm_backward(norm(**kw), qm.LayerNormGradParams(**g), ws, ws_bytes, None)
    assert qm.lib().moe_layer_norm_backward(norm(), None, P, 1 << 30, None) == INVALID
    for g in (dict(dn=None), dict(dx=None), dict(dy=None)):
        assert call(grads=g) == INVALID, g
    assert call(y=None) == INVALID                              # dy without y
    assert call(stats=None) == INVALID
    assert call(ws=None) == INVALID
    for off in (1, 2, 3):
        assert call(ws=P + off) == INVALID
    assert call(ws_bytes=qm.layer_norm_backward_ws_bytes(4, 64) - 1) == WORKSPACE
    assert call(dim=20000) == UNSUPPORTED


@no_gpu
def test_quant_mx_refusals():
    def call(**kw):
        f = dict(x=P, noise=None, q=P, q_scale=P, t=P, t_scale=P, rows=4, cols=70, x_dt=0, q_dt=1, q_layout=0, t_dt=2, t_layout=1)
        f.update(kw)
        return qm.lib().moe_quant_mx(qm.QuantMxParams(**f), None)
    assert qm.lib().moe_quant_mx(None, None) == INVALID
    for bad in (dict(rows=-1), dict(cols=0), dict(x_dt=1), dict(x=None), dict(q=None), dict(t_scale=None), dict(q_dt=0), dict(q_dt=3),
                dict(t_dt=4), dict(q_layout=2), dict(t_layout=-1), dict(q=P + 8), dict(t=P + 4),
                dict(q=None, q_scale=None, t=None, t_scale=None)):
        assert call(**bad) == INVALID, bad
    assert call(q_layout=1) == UNSUPPORTED                      # fp8 has no packed layout
    assert call(t_dt=1) == UNSUPPORTED
    assert call(rows=(1 << 31) - 256, cols=1) == UNSUPPORTED
    assert call(rows=1, cols=(1 << 31) - 1) == UNSUPPORTED
    assert call(rows=1 << 20, cols=1 << 20) == UNSUPPORTED
    assert call(rows=0, x=None) == OK


@no_gpu
def test_pack_mx_refusals():
    Q = P + (1 << 24)
    call = lambda w=P, ws=P + (1 << 20), n=16, k=64, o=Q, os=Q + (1 << 20): qm.lib().moe_pack_mx(w, ws, n, k, o, os, None)   # noqa: E731
    for bad in (dict(w=None), dict(ws=None), dict(o=None), dict(os=None), dict(n=0), dict(k=0), dict(w=P + 8), dict(o=Q + 8),
                dict(o=P), dict(os=P), dict(o=P + (1 << 20)), dict(os=Q)):
        assert call(**bad) == INVALID, bad
    assert call(k=48) == UNSUPPORTED
    assert call(n=1 << 20, k=1 << 14) == UNSUPPORTED


@no_gpu
def test_gemm_mx_refusals():
    def call(a=P, sa=P, dt=1, w=P, ws=P, t=4, n=64, k=128, act=None, add=None, out=P, odt=0):
        return qm.lib().moe_gemm_mx(a, sa, dt, w, ws, t, n, k, act, add, out, odt, None)
    for bad in (dict(t=-1), dict(n=0), dict(k=0), dict(dt=0), dict(dt=4), dict(odt=1), dict(a=None), dict(sa=None), dict(w=None),
                dict(ws=None), dict(out=None), dict(a=P + 8), dict(w=P + 8), dict(sa=P + 2), dict(ws=P + 1),
                dict(act=qm.ActParams(0, 4.0, NAN)), dict(act=qm.ActParams(0, 0.0, 25.0)), dict(act=qm.ActParams(0, INF, 25.0))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(k=64), dict(k=192), dict(k=1 << 24), dict(t=1 << 24), dict(act=qm.ActParams(2, 4.0, 25.0)),
                dict(n=48, act=qm.ActParams(1, 0.0, 0.0)), dict(n=1 << 20, k=1 << 13), dict(t=(1 << 24) - 1, n=1 << 17)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(t=0, a=None) == OK


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(qm, "_on_gpu", lambda t, name: (t.device, t.get_device()))
    monkeypatch.setattr(qm, "_call", lambda fn, *args: pytest.fail(f"{fn} was called"))
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x, w = torch.zeros(4, 128, dtype=bf), torch.ones(128)
    wide = lambda *s, d=bf: torch.empty(*s, dtype=d, device="meta")   # noqa: E731
    big = (1 << 32) + 16
    codes, scale = torch.zeros(4, 128, dtype=u8), torch.zeros(4, 4, dtype=u8)
    pw, ps = (torch.zeros(s, dtype=u8) for s in qm.mx_shapes(64, 128, qm.DT_FP4, True))
    for match, call in (
            ("x", lambda: qm.moe_layer_norm(x.half())), ("x", lambda: qm.moe_layer_norm(x[0])),
            ("strided", lambda: qm.moe_layer_norm(x[:, ::2])), ("y", lambda: qm.moe_layer_norm(x, x.float())),
            ("w", lambda: qm.moe_layer_norm(x, w=w.bfloat16())), ("b:", lambda: qm.moe_layer_norm(x, b=w[:5])),
            ("q_dtype", lambda: qm.moe_layer_norm(x, q_dtype="bf16")), ("h", lambda: qm.moe_layer_norm(x, h=x.float())),
            ("stats", lambda: qm.moe_layer_norm_backward(x, None, torch.zeros(2, 5), x, x)),
            ("dn", lambda: qm.moe_layer_norm_backward(x, None, torch.zeros(2, 4), x, None)),
            ("dh", lambda: qm.moe_layer_norm_backward(x, None, torch.zeros(2, 4), x.float(), x)),
            ("32 bits", lambda: qm.moe_layer_norm(wide(big, 1))), ("32 bits", lambda: qm.moe_layer_norm(wide(1, big))),
            ("x", lambda: qm.moe_quant_mx(x.half(), "fp8")), ("q_dtype", lambda: qm.moe_quant_mx(x, "i8")),
            ("t_dtype", lambda: qm.moe_quant_mx(x)), ("noise", lambda: qm.moe_quant_mx(x, "fp8", noise=codes[:3])),
            ("strided", lambda: qm.moe_quant_mx(x.t(), "fp8")),
            ("32 bits", lambda: qm.moe_quant_mx(wide(big, 1), "fp8")), ("32 bits", lambda: qm.moe_quant_mx(wide(1, big), "fp8")),
            ("w_scale", lambda: qm.moe_pack_mx(codes, scale)), ("w", lambda: qm.moe_pack_mx(codes[0], scale)),
            ("32 bits", lambda: qm.moe_pack_mx(wide(big, 16, d=u8), scale)),
            ("a_dtype", lambda: qm.moe_gemm_mx(codes, scale, "bf16", pw, ps, 64)),
            ("a_scale", lambda: qm.moe_gemm_mx(codes, scale[:, :3], "fp8", pw, ps, 64)),
            ("w", lambda: qm.moe_gemm_mx(codes, torch.zeros(4, 8, dtype=u8), "fp4", pw, ps, 64)),   # 256 columns
            ("w", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps, 65)),
            ("w_scale", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps[:3], 64)),
            ("SiTUv2", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps, 64, act="situv2")),
            ("act", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps, 64, act="gelu")),
            ("out_dtype", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps, 64, out_dtype=torch.float16)),
            ("add", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps, 64, add=torch.zeros(4, 64, dtype=f32))),
            ("32 bits", lambda: qm.moe_gemm_mx(wide(big, 128, d=u8), scale, "fp8", pw, ps, 64)),
            ("32 bits", lambda: qm.moe_gemm_mx(codes, scale, "fp8", pw, ps, big))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(ValueError, match="GPU"):
        monkeypatch.undo()
        qm.moe_layer_norm(x)


@no_gpu
def test_routed_few_refusals():
    silu = qm.ActParams(1, 0.0, 0.0)

    def call(x=P, xs=None, dt=0, w=P, s=P, begin=0, local=8, d=128, i=128, act=silu, out=P, ws=P, ws_bytes=1 << 30, null=False, **kw):
        f = dict(logits=P, bias=None, valid=None, topk_ids=P, topk_w=P, tokens=4, num_experts=8, topk=2, dt=0, score=0, renorm=1, scale=1.0)
        f.update(kw)
        r = None if null else qm.RouterParams(**f)
        return qm.lib().moe_routed_few(r, x, xs, dt, w, s, w, s, begin, local, d, i, act, out, ws, ws_bytes, None)
    for bad in (dict(null=True), dict(tokens=-1), dict(topk=0), dict(num_experts=0), dict(score=2), dict(renorm=2), dict(scale=NAN),
                dict(logits=None), dict(topk_ids=None), dict(topk_w=None), dict(x=None), dict(w=None), dict(s=None), dict(out=None),
                dict(ws=None), dict(dt=3), dict(dt=1), dict(xs=P), dict(act=None), dict(act=qm.ActParams(0, 4.0, INF)), dict(local=0),
                dict(d=0), dict(i=-128), dict(x=P + 8), dict(w=P + 4), dict(s=P + 2), dict(out=P + 2), dict(ws=P + 16),
                dict(dt=2, xs=P + 1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(tokens=17), dict(topk=9), dict(num_experts=2049), dict(local=9), dict(d=192), dict(i=64), dict(d=1 << 24),
                dict(i=1 << 20), dict(act=qm.ActParams(2, 4.0, 25.0))):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(ws_bytes=qm.routed_few_ws_bytes(4, 2, 8, 128, 128, 0) - 1) == WORKSPACE
    assert call(tokens=0, x=None) == OK


def test_routed_few_workspace_matches_the_header(tmp_path):
    cases = [(1, 16, 896, 3584, 384, 0), (16, 16, 896, 3584, 384, 1), (3, 6, 4, 896, 256, 2), (16, 32, 2048, 128, 128, 0), (0, 4, 8, 128, 128, 0)]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "moe_mi355x.h"\nint main(void) {'
                   + "".join('printf("%%zu\\n", moe_routed_few_ws_bytes(%d, %d, %d, %d, %d, %d));' % c for c in cases)
                   + 'printf("%d\\n", MOE_FEW_MAX_TOKENS); return 0; }')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-O1", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [qm.routed_few_ws_bytes(*c) for c in cases] + [qm.FEW_MAX_TOKENS]


def test_routed_few_binding_refusals(monkeypatch):
    monkeypatch.setattr(qm, "_on_gpu", lambda t, name: (t.device, t.get_device()))
    monkeypatch.setattr(qm, "_call", lambda fn, *args: pytest.fail(f"{fn} was called"))
    u8 = torch.uint8
    good = dict(logits=torch.zeros(2, 8), x=torch.zeros(2, 128, dtype=torch.bfloat16), x_scale=None, a_dtype="bf16",
                w1=torch.zeros(8, 256, 64, dtype=u8), w1_scale=torch.zeros(8, 256, 4, dtype=u8),
                w2=torch.zeros(8, 128, 64, dtype=u8), w2_scale=torch.zeros(8, 128, 4, dtype=u8), topk=2, act="silu")
    for match, kw in (("logits", dict(logits=torch.zeros(17, 8))), ("logits", dict(logits=torch.zeros(2, 8, dtype=torch.float16))),
                      ("x:", dict(x=torch.zeros(2, 128))), ("x:", dict(x=torch.zeros(3, 128, dtype=torch.bfloat16))),
                      ("a_dtype", dict(a_dtype="i8")), ("x_scale", dict(x_scale=torch.zeros(2, 4, dtype=u8))),
                      ("x_scale", dict(a_dtype="fp8", x=torch.zeros(2, 128, dtype=u8))), ("w1:", dict(w1=torch.zeros(8, 128, 64, dtype=u8))),
                      ("w1 and w2", dict(w1=torch.zeros(256, 64, dtype=u8))), ("w2_scale", dict(w2_scale=torch.zeros(8, 128, 3, dtype=u8))),
                      ("act", dict(act="gelu")), ("SiTUv2", dict(act="situv2")), ("score", dict(score="relu")),
                      ("out", dict(out=torch.zeros(2, 128))), ("bias", dict(bias=torch.zeros(7))), ("32 bits", dict(topk=1 << 33)),
                      ("32 bits", dict(expert_begin=1 << 31))):
        with pytest.raises(ValueError, match=match):
            qm.moe_routed_few(**{**good, **kw})
