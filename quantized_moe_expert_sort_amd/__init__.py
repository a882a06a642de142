"""Python binding of libmoe_mi355x.so, the gfx950 fused MXFP4 MoE (see include/moe_mi355x.h).

Argument marshalling only: tensors are allocated with torch on the current CUDA (HIP) device,
their data pointers and torch's current stream are passed to the C entry points, and every
step of the operator runs in the library's HIP kernels.  If the library is not built the
calls raise; there is no fallback path.
"""
import collections
import ctypes
import os

import torch

DT_BF16, DT_FP8, DT_FP4 = 0, 1, 2
ACT_SITUV2, ACT_SILU, ACT_NONE_TEST = 0, 1, 2
STAGE_1, STAGE_2, STAGE_ALL = 1, 2, 3
W_ROW_MAJOR, W1_PACKED, W_PACKED = 0, 1, 2
DT_F32, DT_I8 = 3, 4
DTYPES = {"bf16": DT_BF16, "fp8": DT_FP8, "fp4": DT_FP4}
ACTS = {"situv2": ACT_SITUV2, "silu": ACT_SILU, "none_test": ACT_NONE_TEST}

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CAPACITY",
          4: "MOE_ERR_HIP", 5: "MOE_ERR_WORKSPACE", 6: "MOE_ERR_DEBUG_CHECK"}
SORT_CHUNK = 4096
SORT_MIN_CHUNK = 1024

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")
# the same library built with MOE_DEBUG_CHECKS (device-side index checks; every call waits for
# the device and returns MOE_ERR_DEBUG_CHECK when a check failed)
DEBUG_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x_debug.so")
EXPORTS = ("moe_sort", "moe_quant_act", "moe_pack_w1", "moe_pack_w2", "moe_fused", "moe_fused_noalloc",
           "moe_block_norm", "moe_block_norm_backward", "moe_router", "moe_router_backward", "moe_quant_i8",
           "moe_pack_i8", "moe_gemm_i8", "moe_last_hip_error")
NOALLOC_SCRATCH_BYTES = 128 << 20


class MoeError(RuntimeError):
    def __init__(self, fn, status, hip_error=0):
        self.status = status
        msg = f"{fn} returned {STATUS.get(status, status)}"
        if status == 4:
            msg += f" (hipError_t {hip_error})"
        super().__init__(msg)


class Layout(ctypes.Structure):
    _fields_ = [("sorted_token_ids", ctypes.c_void_p), ("sorted_weights", ctypes.c_void_p),
                ("expert_ids", ctypes.c_void_p), ("num_tiles", ctypes.c_void_p),
                ("row_of", ctypes.c_void_p), ("sync", ctypes.c_void_p), ("cap_tiles", ctypes.c_int32),
                ("block_m", ctypes.c_int32)]


class ActParams(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("beta", ctypes.c_float), ("linear_beta", ctypes.c_float)]


class BlockNormParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "y", "w_post", "gate", "w_pre", "h", "n", "q", "q_scale", "rstd")]
                + [(n, ctypes.c_int32) for n in ("tokens", "dim", "x_dt", "gate_kind", "gate_act", "q_dt")]
                + [("scale", ctypes.c_float), ("eps", ctypes.c_float)])


class BlockNormGradParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dh", "dn", "dx", "dy", "dgate", "dw_post", "dw_pre")]


class RouterParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("logits", "bias", "valid", "topk_ids", "topk_w")]
                + [(n, ctypes.c_int32) for n in ("tokens", "num_experts", "topk", "dt", "score", "renorm")]
                + [("scale", ctypes.c_float)])


class BalanceParams(ctypes.Structure):
    _fields_ = ([("coef", ctypes.c_float), ("z_coef", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("counts", "mean_prob", "loss", "num_valid")])


_lib = None


def lib():
    """Load libmoe_mi355x.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run: python -m quantized_moe_expert_sort_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.moe_sort.argtypes = [vp, vp, i32, i32, i32, i32, ctypes.POINTER(Layout), vp, sz, vp]
        L.moe_sort.restype = i32
        L.moe_quant_act.argtypes = [vp, i64, i64, i32, vp, vp, vp]
        L.moe_quant_act.restype = i32
        L.moe_fused.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, vp, ctypes.POINTER(Layout), i32, i32,
                                i32, i32, i32, ctypes.POINTER(ActParams), vp, vp, sz, i32, vp]
        L.moe_fused.restype = i32
        L.moe_fused_noalloc.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, vp, ctypes.POINTER(Layout), i32, i32,
                                        i32, i32, i32, ctypes.POINTER(ActParams), vp, i32, vp]
        L.moe_fused_noalloc.restype = i32
        L.moe_pack_w1.argtypes = [vp, i32, i32, i32, vp, vp]
        L.moe_pack_w1.restype = i32
        L.moe_pack_w2.argtypes = [vp, i32, i32, i32, vp, vp]
        L.moe_pack_w2.restype = i32
        L.moe_block_norm.argtypes = [ctypes.POINTER(BlockNormParams), vp]
        L.moe_block_norm.restype = i32
        L.moe_block_norm_backward.argtypes = [ctypes.POINTER(BlockNormParams), ctypes.POINTER(BlockNormGradParams), vp,
                                              sz, vp]
        L.moe_block_norm_backward.restype = i32
        L.moe_router.argtypes = [ctypes.POINTER(RouterParams), ctypes.POINTER(BalanceParams), vp, sz, vp]
        L.moe_router.restype = i32
        L.moe_router_backward.argtypes = [ctypes.POINTER(RouterParams), ctypes.POINTER(BalanceParams), vp, vp, vp, vp]
        L.moe_router_backward.restype = i32
        L.moe_quant_i8.argtypes = [vp, i64, i64, vp, vp, vp]
        L.moe_quant_i8.restype = i32
        L.moe_pack_i8.argtypes = [vp, i32, i32, vp, vp]
        L.moe_pack_i8.restype = i32
        L.moe_gemm_i8.argtypes = [vp, vp, vp, vp, i32, i32, i32, ctypes.POINTER(ActParams), vp, vp, vp]
        L.moe_gemm_i8.restype = i32
        L.moe_last_hip_error.argtypes = []
        L.moe_last_hip_error.restype = i32
        _lib = L
    return _lib


def select_library(path):
    """Route later calls to the library at `path` (LIB_PATH or DEBUG_LIB_PATH); returns the
    previous path."""
    global LIB_PATH, _lib
    prev, LIB_PATH, _lib = LIB_PATH, path, None
    return prev


def _check(fn, status):
    if status != 0:
        raise MoeError(fn, status, lib().moe_last_hip_error() if status == 4 else 0)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


# ------------------------------------------------------------------ size helpers (mirror the
# static inline helpers of include/moe_mi355x.h)

def _align256(b):
    return (b + 255) & ~255


def block_m(tokens):
    """Rows per tile the kernels are tuned for (moe_block_m of the header)."""
    return 16 if tokens <= 512 else 32


def cap_tiles(tokens, topk, num_local_experts, block_m):
    n = tokens * topk
    return (n + block_m - 1) // block_m + min(num_local_experts, n)


SINGLE_LAUNCH_MAX_TOKENS = 2048
SYNC_CLASSES = 16


def sync_words(tokens, cap):
    return 16 * (1 + 2 * cap + SYNC_CLASSES * tokens)


def sort_ws_bytes(tokens, topk, num_local_experts):
    n = tokens * topk
    chunks = (n + SORT_MIN_CHUNK - 1) // SORT_MIN_CHUNK
    return _align256((chunks + 2) * num_local_experts * 4) + _align256(n * 4)


def row_bytes(cols, dt):
    return cols * 2 if dt == DT_BF16 else cols if dt == DT_FP8 else cols // 2


def rowout_elem_bytes(a_dtype):
    return 2


HOT_MAX = 16
WS_PARTS = ("rowout", "inter", "iscale", "groups", "cgroups", "tile_hot", "hot_e", "hotpos", "hotw", "hotmask",
            "hot_out", "dbg", "total")


def fused_ws_parts(tokens, model_dim, inter_dim, cap, block_m, a_dtype, act):
    """Byte offsets of the workspace parts and the total (moe_fused_ws_parts of the header)."""
    rows = cap * block_m
    t = max(tokens, 0)
    sizes = [_align256(rows * model_dim * rowout_elem_bytes(a_dtype)),
             _align256((rows + 1) * row_bytes(inter_dim, a_dtype)),
             _align256(0 if a_dtype == DT_BF16 else (rows + 1) * (inter_dim // 32)),
             _align256(cap * 8) + 256, _align256(cap * 8) + 256, _align256(cap * 4), 256,
             _align256(t * HOT_MAX * 4), _align256(t * HOT_MAX * 4), _align256(t * 4),
             _align256(t * model_dim * 2),
             _align256(rows * inter_dim * 2 * 4) if act == ACT_NONE_TEST else 0]
    out, o = {}, 0
    for name, sz in zip(WS_PARTS, sizes):
        out[name] = o
        o += sz
    out["total"] = o
    return out


def fused_debug_offset(tokens, model_dim, inter_dim, cap, block_m, a_dtype):
    return fused_ws_parts(tokens, model_dim, inter_dim, cap, block_m, a_dtype, ACT_NONE_TEST)["dbg"]


def fused_ws_bytes(tokens, model_dim, inter_dim, cap, block_m, a_dtype, act):
    return fused_ws_parts(tokens, model_dim, inter_dim, cap, block_m, a_dtype, act)["total"]


# ------------------------------------------------------------------ entry points

class MoeLayout:
    """Device buffers of a sorted layout (owned by torch) plus its ctypes view."""

    def __init__(self, tokens, topk, num_local_experts, block_m, with_weights=True, device="cuda",
                 cap=None, single_launch=False):
        """single_launch: allocate the sync words that let moe_fused run batches below
        SINGLE_LAUNCH_MAX_TOKENS as one launch (False: one launch per stage)."""
        self.block_m = block_m
        self.cap = cap_tiles(tokens, topk, num_local_experts, block_m) if cap is None else cap
        n = max(self.cap * block_m, 1)
        self.sorted_token_ids = torch.empty(n, dtype=torch.int32, device=device)
        self.sorted_weights = torch.empty(n, dtype=torch.float32, device=device) if with_weights else None
        self.expert_ids = torch.empty(max(self.cap, 1), dtype=torch.int32, device=device)
        self.num_tiles = torch.empty(1, dtype=torch.int32, device=device)
        self.row_of = torch.empty(max(tokens * topk, 1), dtype=torch.int32, device=device)
        self.sync = (torch.empty(sync_words(tokens, self.cap), dtype=torch.int32, device=device)
                     if single_launch else None)
        self.c = Layout(self.sorted_token_ids.data_ptr(),
                        None if self.sorted_weights is None else self.sorted_weights.data_ptr(),
                        self.expert_ids.data_ptr(), self.num_tiles.data_ptr(), self.row_of.data_ptr(),
                        None if self.sync is None else self.sync.data_ptr(), self.cap, block_m)


def moe_sort(topk_ids, topk_w, expert_begin, num_local_experts, block_m, with_weights=True,
             layout=None, ws=None, single_launch=False):
    """Route-sort on the GPU; returns a MoeLayout (see moe_sort in the header)."""
    T, K = topk_ids.shape
    if layout is None:
        layout = MoeLayout(T, K, num_local_experts, block_m, with_weights, topk_ids.device,
                           single_launch=single_launch)
    if ws is None:
        ws = torch.empty(max(sort_ws_bytes(T, K, num_local_experts), 1), dtype=torch.uint8,
                         device=topk_ids.device)
    _check("moe_sort", lib().moe_sort(_ptr(topk_ids), _ptr(topk_w) if with_weights else None, T, K,
                                      expert_begin, num_local_experts, ctypes.byref(layout.c),
                                      _ptr(ws), ws.numel(), _stream()))
    return layout


def moe_pack_w1(w1, out=None):
    """Stage1 weights [E, 2I, D/2] uint8 (row-major) -> the packed layout moe_fused reads."""
    E, rows, half_d = w1.shape
    if out is None:
        out = torch.empty_like(w1)
    _check("moe_pack_w1", lib().moe_pack_w1(_ptr(w1), E, half_d * 2, rows // 2, _ptr(out), _stream()))
    return out


def moe_pack_w2(w2, out=None):
    """Stage2 weights [E, D, I/2] uint8 (row-major) -> the packed layout moe_fused reads."""
    E, D, half_i = w2.shape
    if out is None:
        out = torch.empty_like(w2)
    _check("moe_pack_w2", lib().moe_pack_w2(_ptr(w2), E, D, half_i * 2, _ptr(out), _stream()))
    return out


def device_weights(w1, w1s, w2, w2s, device="cuda"):
    """Host MXFP4 weights (numpy, row-major) -> the device tuple moe_fused takes (w1 and w2
    packed, the scales as they are)."""
    w1_d, w1s_d, w2_d, w2s_d = (torch.from_numpy(a).to(device) for a in (w1, w1s, w2, w2s))
    p1, p2 = moe_pack_w1(w1_d), moe_pack_w2(w2_d)
    del w1_d, w2_d
    return p1, w1s_d, p2, w2s_d


def moe_quant_act(x_bf16, dt, q=None, scale=None):
    """bf16 [rows, cols] -> (codes, e8m0 scales); dt is "fp8" or "fp4"."""
    d = DTYPES[dt] if isinstance(dt, str) else dt
    rows, cols = x_bf16.shape
    if q is None:
        q = torch.empty((rows, cols if d == DT_FP8 else cols // 2), dtype=torch.uint8, device=x_bf16.device)
    if scale is None:
        scale = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x_bf16.device)
    _check("moe_quant_act", lib().moe_quant_act(_ptr(x_bf16), rows, cols, d, _ptr(q), _ptr(scale), _stream()))
    return q, scale


def moe_fused(x, x_scale, a_dtype, w1, w1_scale, w2, w2_scale, topk_w, layout, num_local_experts,
              act="situv2", beta=None, linear_beta=None, out=None, ws=None, stages=STAGE_ALL,
              w_layout=W_PACKED):
    """Stage1 + Stage2 over a layout from moe_sort; returns out [T, D] bf16 (or, for
    act="none_test", the workspace tensor holding the raw gate/up sums).  w1 and w2 are in the
    layout named by w_layout (the library reads W_PACKED, as moe_pack_w1 / moe_pack_w2 write
    them; device_weights does both).  stages selects
    STAGE_1, STAGE_2 (reusing the intermediate a STAGE_1 call left in the same ws) or both."""
    d = DTYPES[a_dtype] if isinstance(a_dtype, str) else a_dtype
    a = ACTS[act] if isinstance(act, str) else act
    T, K = topk_w.shape
    D = w2.shape[1]
    I = w2.shape[2] * 2
    if a == ACT_SITUV2 and (beta is None or linear_beta is None):
        raise ValueError("SiTUv2 needs beta and linear_beta (there are no defaults)")
    params = ActParams(a, 0.0 if beta is None else beta, 0.0 if linear_beta is None else linear_beta)
    if ws is None:
        ws = torch.empty(fused_ws_bytes(T, D, I, layout.cap, layout.block_m, d, a), dtype=torch.uint8,
                         device=topk_w.device)
    if out is None and a != ACT_NONE_TEST:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=topk_w.device)
    _check("moe_fused", lib().moe_fused(_ptr(x), _ptr(x_scale), d, _ptr(w1), w_layout, _ptr(w1_scale), _ptr(w2),
                                        _ptr(w2_scale), _ptr(topk_w), ctypes.byref(layout.c), T, K,
                                        num_local_experts, D, I, ctypes.byref(params), _ptr(out),
                                        _ptr(ws), ws.numel(), stages, _stream()))
    return ws if a == ACT_NONE_TEST else out


def moe_fused_noalloc(x, x_scale, a_dtype, w1, w1_scale, w2, w2_scale, topk_w, layout, num_local_experts,
                      act="situv2", beta=None, linear_beta=None, out=None, stages=STAGE_ALL,
                      w_layout=W_PACKED):
    """moe_fused with the library's fixed per-device scratch as its workspace (nothing allocated
    for the workspace; calls on one device share it and must not overlap).  Returns out."""
    d = DTYPES[a_dtype] if isinstance(a_dtype, str) else a_dtype
    a = ACTS[act] if isinstance(act, str) else act
    T, K = topk_w.shape
    D = w2.shape[1]
    I = w2.shape[2] * 2
    if a == ACT_SITUV2 and (beta is None or linear_beta is None):
        raise ValueError("SiTUv2 needs beta and linear_beta (there are no defaults)")
    params = ActParams(a, 0.0 if beta is None else beta, 0.0 if linear_beta is None else linear_beta)
    if out is None and a != ACT_NONE_TEST:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=topk_w.device)
    _check("moe_fused_noalloc", lib().moe_fused_noalloc(_ptr(x), _ptr(x_scale), d, _ptr(w1), w_layout,
                                                        _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), _ptr(topk_w),
                                                        ctypes.byref(layout.c), T, K, num_local_experts, D, I,
                                                        ctypes.byref(params), _ptr(out), stages, _stream()))
    return out


# ------------------------------------------------------------------ around the routed experts
#
# These check their tensors (type, shape, dense rows, one device) before the C call checks the
# rest, and run on the device of their first tensor, on torch's current stream of that device.

NORM_MAX_DIM, NORM_PARTS = 16384, 256
GATES = {"none": 0, "channel": 1, "token": 2, "element": 3}
GATE_ACTS = {"none": 0, "sigmoid": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
ROUTER_MAX_TOPK, ROUTER_PARTS = 32, 256
Q_DTYPES = {"fp8": DT_FP8, "fp4": DT_FP4, "i8": DT_I8}
_ROW_TYPES = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}

BlockNorm = collections.namedtuple("BlockNorm", "h n q q_scale rstd")
BlockNormGrads = collections.namedtuple("BlockNormGrads", "dx dy dgate dw_post dw_pre")
Routing = collections.namedtuple("Routing", "ids w balance")
Balance = collections.namedtuple("Balance", "counts mean_prob loss num_valid coef z_coef")


def block_norm_backward_ws_bytes(tokens, dim):
    return _align256(min(max(tokens, 0), NORM_PARTS) * 3 * dim * 4)


def router_ws_bytes(num_experts):
    return 512 + 8 * ROUTER_PARTS + _align256(ROUTER_PARTS * num_experts * 8)


def i8_packed_shape(out_features, in_features):
    """Shape of moe_pack_i8's result: 1 KB blocks of 16 rows x 64 bytes."""
    return ((out_features + 15) // 16, (in_features + 127) // 128 * 2, 1024)


def _need(t, name, dtype, shape, index):
    """The tensor's address (None for None), after its checks; index: the device's."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: need a dense {dtype} tensor of shape {tuple(shape)} on device {index}, got "
                     f"{'a dense' if t.is_contiguous() else 'a strided'} {t.dtype} of {tuple(t.shape)} on {t.device}")


def _sizes(*values):
    """Refuses sizes that the library's 32-bit arguments cannot hold (ctypes would wrap them)."""
    if max(values) > 0x7FFFFFFF or min(values) < -0x80000000:
        raise ValueError(f"sizes have to fit 32 bits, got {', '.join(map(str, values))}")


def _pick(table, key, name):
    if key not in table:
        raise ValueError(f"{name}: {key!r} is none of {', '.join(table)}")
    return table[key]


# torch's getters without their lazy-initialisation wrappers, where this build of torch has them: a
# call's tensors are on the GPU already (2.7 us less of a call's 12 us on the host)
def _public_device():
    return torch.cuda.current_device()


def _public_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", _public_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)


def _call(fn, index, *args):
    """The library call on torch's current stream of device `index`, with that device current."""
    f = getattr(_lib or lib(), fn)
    if index == _current_device():
        status = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = f(*args, _raw_stream(index))
    if status:
        _check(fn, status)


def _on_gpu(t, name):
    """(device, its index) of a tensor that has to be on the GPU."""
    if not t.is_cuda:
        raise ValueError(f"{name}: need a tensor on the GPU, got one on {t.device}")
    return t.device, t.get_device()


def _norm_params(x, y, w_post, gate, gate_kind, gate_act, scale, w_pre, eps, index):
    if x.dim() != 2 or x.dtype not in _ROW_TYPES:
        raise ValueError(f"x: need a bfloat16 or float32 tensor [tokens, dim], got {x.dtype} of {tuple(x.shape)}")
    T, D = x.shape
    _sizes(T, D)
    kind = _pick(GATES, gate_kind, "gate_kind")
    if (gate is None) != (kind == 0):
        raise ValueError("gate and gate_kind go together")
    p = BlockNormParams(tokens=T, dim=D, x_dt=_ROW_TYPES[x.dtype], gate_kind=kind,
                        gate_act=_pick(GATE_ACTS, gate_act, "gate_act"), scale=scale, eps=eps)
    p.x = _need(x, "x", x.dtype, (T, D), index)
    p.y = _need(y, "y", torch.bfloat16, (T, D), index)
    p.w_post = _need(w_post, "w_post", torch.float32, (D,), index)
    p.w_pre = _need(w_pre, "w_pre", torch.float32, (D,), index)
    if kind:
        p.gate = _need(gate, "gate", torch.bfloat16 if kind == 3 else torch.float32,
                       ((D,), (T,), (T, D))[kind - 1], index)
    return p, T, D


def moe_block_norm(x, y=None, *, w_post=None, gate=None, gate_kind="none", gate_act="none", scale=1.0, w_pre=None,
                   eps=1e-6, h=None, want_n=True, q_dtype=None, stats=False):
    """The norm after a block, its gate, the residual sum and the norm before the next block (see
    moe_block_norm in the header).  x bf16 or fp32 [T, D], y bf16 [T, D], weights fp32 [D].

    Returns BlockNorm(h, n, q, q_scale, rstd): h as x (None without y; pass h=x to update the stream in
    place), n bf16 (None without w_pre or with want_n=False), q and q_scale for q_dtype "fp8", "fp4" or
    "i8", rstd [2, T] with stats=True (the backward pass needs it)."""
    device, index = _on_gpu(x, "x")
    p, T, D = _norm_params(x, y, w_post, gate, gate_kind, gate_act, scale, w_pre, eps, index)
    n = q = q_scale = rstd = None
    if h is not None:
        p.h = _need(h, "h", x.dtype, (T, D), index)
    elif y is not None:
        h = torch.empty_like(x)
        p.h = h.data_ptr()
    if w_pre is not None and want_n:
        n = torch.empty(T, D, dtype=torch.bfloat16, device=device)
        p.n = n.data_ptr()
    if q_dtype is not None:
        p.q_dt = _pick(Q_DTYPES, q_dtype, "q_dtype")
        if w_pre is None:
            raise ValueError("q_dtype: there is nothing to code without w_pre")
        if p.q_dt == DT_I8:
            q = torch.empty(T, D, dtype=torch.int8, device=device)
            q_scale = torch.empty(T, dtype=torch.float32, device=device)
        else:
            q = torch.empty(T, D if p.q_dt == DT_FP8 else D // 2, dtype=torch.uint8, device=device)
            q_scale = torch.empty(T, D // 32, dtype=torch.uint8, device=device)
        p.q, p.q_scale = q.data_ptr(), q_scale.data_ptr()
    if stats:
        rstd = torch.empty(2, T, dtype=torch.float32, device=device)
        p.rstd = rstd.data_ptr()
    _call("moe_block_norm", index, p)
    return BlockNorm(h, n, q, q_scale, rstd)


def moe_block_norm_backward(x, y, rstd, dh, dn, *, w_post=None, gate=None, gate_kind="none", gate_act="none",
                            scale=1.0, w_pre=None, dx=None, ws=None):
    """Gradients of moe_block_norm for its inputs, from those of h (dh, as x) and n (dn, bf16); either
    may be None.  rstd: as moe_block_norm(stats=True) returned it; the other arguments as given there.
    dx: where its gradient goes (as x), which may be dh, or None for a new tensor.
    Returns BlockNormGrads(dx, dy, dgate, dw_post, dw_pre), None for what was not given."""
    device, index = _on_gpu(x, "x")
    p, T, D = _norm_params(x, y, w_post, gate, gate_kind, gate_act, scale, w_pre, 1.0, index)
    p.rstd = _need(rstd, "rstd", torch.float32, (2, T), index)
    g = BlockNormGradParams()
    g.dh = _need(dh, "dh", x.dtype, (T, D), index)
    g.dn = _need(dn, "dn", torch.bfloat16, (T, D), index)
    dy = dgate = dw_post = dw_pre = None
    if dx is None:
        dx = torch.empty_like(x)
    g.dx = _need(dx, "dx", x.dtype, (T, D), index)
    if y is not None:
        dy = torch.empty_like(y)
        g.dy = dy.data_ptr()
    if gate is not None:
        dgate = torch.empty_like(gate)
        g.dgate = dgate.data_ptr()
    if w_post is not None:
        dw_post = torch.empty_like(w_post)
        g.dw_post = dw_post.data_ptr()
    if dn is not None:
        dw_pre = torch.empty(D, dtype=torch.float32, device=device)
        g.dw_pre = dw_pre.data_ptr()
    if ws is None:
        ws = torch.empty(block_norm_backward_ws_bytes(T, D), dtype=torch.uint8, device=device)
    _call("moe_block_norm_backward", index, p, g, _need(ws, "ws", torch.uint8, ws.shape, index), ws.numel())
    return BlockNormGrads(dx, dy, dgate, dw_post, dw_pre)


def _router_params(logits, topk, score, renorm, scale, bias, valid, index):
    if logits.dim() != 2 or logits.dtype not in _ROW_TYPES:
        raise ValueError(f"logits: need a bfloat16 or float32 tensor [tokens, experts], got {logits.dtype} of "
                         f"{tuple(logits.shape)}")
    T, E = logits.shape
    _sizes(T, E, topk)
    if valid is not None and valid.dtype == torch.bool:
        valid = valid.view(torch.uint8)
    r = RouterParams(tokens=T, num_experts=E, topk=topk, dt=_ROW_TYPES[logits.dtype],
                     score=_pick(SCORES, score, "score"), renorm=int(bool(renorm)), scale=scale)
    r.logits = _need(logits, "logits", logits.dtype, (T, E), index)
    r.bias = _need(bias, "bias", torch.float32, (E,), index)
    r.valid = _need(valid, "valid", torch.uint8, (T,), index)
    return r, T, E


def moe_router(logits, topk, *, score="softmax", renorm=True, scale=1.0, bias=None, valid=None, balance=None, ws=None):
    """The topk experts of each token and their weights, as moe_sort and moe_fused take them (see
    moe_router in the header).  logits bf16 or fp32 [T, E]; bias fp32 [E], for the choice only; valid
    bool or uint8 [T], 0 for padding; balance: (coef, z_coef) to take the balance loss, the z loss and
    the per-expert counts in the same pass.

    Returns Routing(ids int32 [T, topk], w fp32 [T, topk], balance), balance being None or
    Balance(counts, mean_prob, loss [2], num_valid, coef, z_coef)."""
    device, index = _on_gpu(logits, "logits")
    r, T, E = _router_params(logits, topk, score, renorm, scale, bias, valid, index)
    ids = torch.empty(T, max(topk, 0), dtype=torch.int32, device=device)
    w = torch.empty(T, max(topk, 0), dtype=torch.float32, device=device)
    r.topk_ids, r.topk_w = ids.data_ptr(), w.data_ptr()
    if balance is None:
        _call("moe_router", index, r, None, None, 0)
        return Routing(ids, w, None)
    coef, z_coef = balance
    b = Balance(torch.empty(E, dtype=torch.int32, device=device), torch.empty(E, dtype=torch.float32, device=device),
                torch.empty(2, dtype=torch.float32, device=device), torch.empty(1, dtype=torch.int32, device=device),
                coef, z_coef)
    if ws is None:
        ws = torch.empty(router_ws_bytes(E), dtype=torch.uint8, device=device)
    _call("moe_router", index, r, _balance_params(b), _need(ws, "ws", torch.uint8, ws.shape, index), ws.numel())
    return Routing(ids, w, b)


def _balance_params(b):
    return BalanceParams(b.coef, b.z_coef, b.counts.data_ptr(), b.mean_prob.data_ptr(), b.loss.data_ptr(),
                         b.num_valid.data_ptr())


def moe_router_backward(logits, routing, d_w=None, *, d_loss=None, score="softmax", renorm=True, scale=1.0, valid=None):
    """d_logits of moe_router, given its result: from d_w (fp32 [T, topk], gradient of the weights) and,
    where it took the balance statistics, d_loss (fp32 [2] on the GPU, gradients of the two losses;
    None for ones).  The other arguments as in the forward call."""
    device, index = _on_gpu(logits, "logits")
    if routing.ids.dim() != 2:
        raise ValueError(f"routing.ids: need [tokens, topk], got {tuple(routing.ids.shape)}")
    topk = routing.ids.shape[1]
    r, T, E = _router_params(logits, topk, score, renorm, scale, None, valid, index)
    r.topk_ids = _need(routing.ids, "routing.ids", torch.int32, (T, topk), index)
    b = routing.balance
    if b is not None:
        _need(b.counts, "balance.counts", torch.int32, (E,), index)
        _need(b.num_valid, "balance.num_valid", torch.int32, (1,), index)
        b = _balance_params(b)
    d_logits = torch.empty_like(logits)
    _call("moe_router_backward", index, r, b, _need(d_w, "d_w", torch.float32, (T, topk), index),
          _need(d_loss, "d_loss", torch.float32, (2,), index), d_logits.data_ptr())
    return d_logits


def moe_quant_i8(x, q=None, scale=None):
    """bf16 [rows, cols] -> (int8 codes, fp32 scale per row), see moe_quant_i8 in the header."""
    device, index = _on_gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: need [rows, cols], got {tuple(x.shape)}")
    rows, cols = x.shape
    if q is None:
        q = torch.empty(rows, cols, dtype=torch.int8, device=device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=device)
    _call("moe_quant_i8", index, _need(x, "x", torch.bfloat16, (rows, cols), index), rows, cols,
          _need(q, "q", torch.int8, (rows, cols), index), _need(scale, "scale", torch.float32, (rows,), index))
    return q, scale


def moe_pack_i8(w, out=None):
    """int8 weights [out_features, in_features] -> the packed layout moe_gemm_i8 reads."""
    device, index = _on_gpu(w, "w")
    if w.dim() != 2:
        raise ValueError(f"w: need [out_features, in_features], got {tuple(w.shape)}")
    N, K = w.shape
    _sizes(N, K)
    shape = i8_packed_shape(N, K)
    if out is None:
        out = torch.empty(shape, dtype=torch.int8, device=device)
    _call("moe_pack_i8", index, _need(w, "w", torch.int8, (N, K), index), N, K,
          _need(out, "out", torch.int8, shape, index))
    return out


def moe_gemm_i8(a, a_scale, w_packed, w_scale, *, act=None, beta=None, linear_beta=None, add=None, out=None):
    """int8 tokens [T, K] (scales [T]) times packed int8 weights of w_scale.numel() rows -> bf16, with
    act "situv2" or "silu" of the [gate|up] halves and `add` (bf16, shape of the result) in the same
    launch (see moe_gemm_i8 in the header)."""
    device, index = _on_gpu(a, "a")
    if a.dim() != 2 or w_scale.dim() != 1:
        raise ValueError(f"need a [tokens, in_features] and w_scale [out_features], got {tuple(a.shape)} and "
                         f"{tuple(w_scale.shape)}")
    T, K = a.shape
    N = w_scale.shape[0]
    _sizes(T, N, K)
    params = None
    if act is not None:
        k = _pick(ACTS, act, "act")
        if k == ACT_SITUV2 and (beta is None or linear_beta is None):
            raise ValueError("SiTUv2 needs beta and linear_beta (there are no defaults)")
        params = ActParams(k, 0.0 if beta is None else beta, 0.0 if linear_beta is None else linear_beta)
    shape = (T, N if act is None else N // 2)
    if out is None:
        out = torch.empty(*shape, dtype=torch.bfloat16, device=device)
    _call("moe_gemm_i8", index, _need(a, "a", torch.int8, (T, K), index),
          _need(a_scale, "a_scale", torch.float32, (T,), index),
          _need(w_packed, "w_packed", torch.int8, i8_packed_shape(N, K), index),
          _need(w_scale, "w_scale", torch.float32, (N,), index), T, N, K, params,
          _need(add, "add", torch.bfloat16, shape, index), _need(out, "out", torch.bfloat16, shape, index))
    return out
