"""B200 (sm_100a) fine-grained MoE layer forward -- Python binding.

A thin ctypes binding over ``libmoe_gate.so`` (the C ABI in
``include/moe_gate.h``): each function has the C entry point's name and
arguments, takes torch tensors (or raw device pointers as ints) and raises
``MoEError`` on a non-OK status.  Every step of the layer runs in the
library's CUDA kernels; PyTorch only provides device memory and streams.
There is no CPU fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gate.so")

MOE_F32, MOE_BF16 = 0, 1

STATUS = {
    0: "MOE_OK",
    1: "MOE_ERR_INVALID_ARG",
    2: "MOE_ERR_UNSUPPORTED",
    3: "MOE_ERR_ALIGNMENT",
    4: "MOE_ERR_WORKSPACE",
    5: "MOE_ERR_CUDA",
    6: "MOE_ERR_DEVICE_CHECK",
    7: "MOE_ERR_TIMEOUT",
}

EXPORTS = (
    "moe_route", "moe_load_and_bias_update", "moe_permute", "moe_permute_workspace_size", "moe_permute_noalloc",
    "moe_grouped_swiglu", "moe_grouped_swiglu_workspace_size", "moe_expert_up", "moe_expert_down", "moe_ffn_up",
    "moe_ffn_down", "moe_ffn_down_combine", "moe_combine_finish", "moe_combine", "moe_layer_forward",
    "moe_workspace_size", "moe_get_last_error",
    "moe_kernel_launch_count", "moe_selftest_bounded_wait", "moe_status_string", "moe_abi_version",
    "moe_quantize_fp8", "moe_fp8_scale_bytes", "moe_fp8_tile_scales", "moe_fp8_tile_scale_bytes", "moe_ffn_up_fp8",
    "moe_ffn_up_fp8_quant", "moe_ffn_down_fp8",
    "moe_layer_forward_fp8",
    "moe_ep_plan_size", "moe_ep_plan", "moe_ep_dispatch", "moe_ep_return",
    "moe_layer_backward", "moe_backward_workspace_size",
    "moe_gate_logits", "moe_route_logits", "moe_route_logits_backward", "moe_ffn_up_save",
    "moe_swiglu_backward_saved",
    "moe_layer_forward_logits", "moe_layer_backward_logits", "moe_backward_logits_workspace_size",
)

MOE_ROUTED, MOE_SHARED = 0, 1
MOE_F32, MOE_BF16, MOE_FP8_E4M3 = 0, 1, 2


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class MoEShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("S", ctypes.c_int32), ("Is", ctypes.c_int32), ("dtype", ctypes.c_int32)]

    def __repr__(self):
        return "MoEShape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def shape_of(cfg, T: int | None = None) -> MoEShape:
    """MoEShape from a workload config (``inputs.MoEConfig``)."""
    return MoEShape(cfg.T if T is None else T, cfg.d, cfg.E, cfg.k, cfg.I, cfg.S, cfg.Is,
                    {"bf16": MOE_BF16, "fp8": MOE_FP8_E4M3}.get(cfg.dtype, MOE_F32))


class MoEFp8Experts(ctypes.Structure):
    """moe_fp8_experts: E4M3 expert weights and their 1x32-tile power-of-two
    scales (W1/W3 scales in one gate/up buffer, W2 in 128-row atoms)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("w1", "w3", "w13_scale", "w2", "w2_scale",
                                               "ws1", "ws3", "ws13_scale", "ws2", "ws2_scale")]


def fp8_experts(q: dict) -> MoEFp8Experts:
    """MoEFp8Experts from a dict of device tensors with keys w1q, w3q, w13s,
    w2q, w2s, ... (the layout of ``quantize_experts_fp8``).  The tensors must
    outlive its use."""
    f = {n: _p(q.get(n + "q")) for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2")}
    for n in ("w13", "w2", "ws13", "ws2"):
        f[n + "_scale"] = _p(q.get(n + "s"))
    return MoEFp8Experts(**f)


MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1


class MoERouteOpts(ctypes.Structure):
    """moe_route_opts: the form of the gate (see moe_gate.h)."""
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


def route_opts(score="sigmoid", groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0) -> MoERouteOpts:
    """MoERouteOpts from plain values; the defaults are moe_route's own gate."""
    kinds = {"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}
    if score not in kinds:
        raise ValueError(f"score must be one of {sorted(kinds)}, got {score!r}")
    return MoERouteOpts(kinds[score], groups, top_groups, group_top, int(bool(renormalize)), scale)


class MoESavedActs(ctypes.Structure):
    """moe_saved_acts: the gate/up pre-activations of a forward in 8 bits."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("a", "a_scale", "g", "g_scale", "sa", "sa_scale", "sg", "sg_scale")]


def saved_acts(t: dict) -> MoESavedActs:
    """MoESavedActs from a dict of device tensors under its field names (the
    layout of ``saved_act_buffers``), or of raw pointers.  It keeps the tensors;
    each call it is passed to checks that they are large enough for its shape."""
    out, device = MoESavedActs(*[_p(t.get(n)) for n, _ in MoESavedActs._fields_]), None
    out.tensors, out.sizes = dict(t), {}
    for n, _ in MoESavedActs._fields_:
        v = t.get(n)
        if v is None or isinstance(v, int):
            continue
        if not v.is_contiguous():
            raise MoEError(1, f"saved_acts: {n} must be contiguous, got strides {v.stride()}")
        if device is not None and device != v.get_device():
            raise MoEError(1, f"saved_acts: {n} must be on one device with the others, got {v.device}")
        device, out.sizes[n] = v.get_device(), _nbytes(v)
    out.device = device  # -1: the CPU, which the calls refuse
    # elements each expert set's buffers hold (a tile of 32 has a scale byte)
    out.room = {pre: min([out.sizes[n] * (32 if n.endswith("scale") else 1) for n in (pre + "a", pre + "a_scale",
                          pre + "g", pre + "g_scale") if n in out.sizes], default=None) for pre in ("", "s")}
    return out


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises MoEError-free ImportError if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m fine_grained_moe_gate_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, S, F = ctypes.c_void_p, MoEShape, ctypes.c_float
        sz = ctypes.c_size_t
        sig = {
            "moe_route": [P, P, P, S, P, P, P, P, P],
            "moe_load_and_bias_update": [P, S, F, P, P, P, P],
            "moe_permute": [P, P, P, S, P, P, P, P, P, sz, P],
            "moe_permute_noalloc": [P, P, P, S, P, P, P, P, P],
            "moe_grouped_swiglu": [P, P, P, P, P, P, P, P, P, S, P, P, P, sz, P],
            "moe_expert_up": [P, P, P, P, P, S, ctypes.c_int32, P, P],
            "moe_expert_down": [P, P, P, S, ctypes.c_int32, P, P],
            "moe_ffn_up": [P, P, P, P, P, P, P, S, P, P, P],
            "moe_ffn_down": [P, P, P, P, P, S, P, P, P],
            "moe_combine": [P, P, P, P, S, P, P],
            "moe_ffn_down_combine": [P, P, P, P, P, P, P, S, P, P],
            "moe_combine_finish": [P, S, P, P],
            "moe_layer_forward": [P, P, P, P, P, P, P, P, P, S, P, P, P, P, P, sz, P],
            "moe_get_last_error": [P],
            "moe_quantize_fp8": [P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P],
            "moe_ffn_up_fp8": [P, P, P, P, P, ctypes.POINTER(MoEFp8Experts), S, P, P, P],
            "moe_ffn_up_fp8_quant": [P, P, P, P, P, ctypes.POINTER(MoEFp8Experts), S, P, P, P, P, P],
            "moe_fp8_tile_scales": [P, ctypes.c_int64, ctypes.c_int32, P, ctypes.c_int32, P, ctypes.c_int32,
                                    ctypes.c_int64, P, P],
            "moe_ffn_down_fp8": [P, P, P, P, P, ctypes.POINTER(MoEFp8Experts), S, P, P, P],
            "moe_layer_forward_fp8": [P, P, P, ctypes.POINTER(MoEFp8Experts), S, P, P, P, P, P, sz, P],
            "moe_ep_plan": [P, ctypes.c_int32, ctypes.c_int32, S, ctypes.c_int64, P, P, P],
            "moe_ep_dispatch": [P, P, P, ctypes.c_int32, ctypes.c_int32, S, P, P],
            "moe_ep_return": [P, P, ctypes.c_int32, ctypes.c_int32, S, P, P],
            "moe_selftest_bounded_wait": [ctypes.c_uint32, P],
            "moe_gate_logits": [P, P, S, P, P],
            "moe_route_logits": [P, P, S, MoERouteOpts, P, P, P, P],
            "moe_route_logits_backward": [P, P, P, P, S, MoERouteOpts, P, P],
            "moe_ffn_up_save": [P, P, P, P, P, P, P, S, P, P, ctypes.POINTER(MoESavedActs), P],
            "moe_swiglu_backward_saved": [ctypes.POINTER(MoESavedActs), S, ctypes.c_int32, P, P, P, P, P, P, P],
            "moe_layer_forward_logits": [P, P, P, P, P, P, P, P, P, S, MoERouteOpts, P, P, P, P, P,
                                         ctypes.POINTER(MoESavedActs), P, sz, P],
            "moe_layer_backward_logits": [P, P, P, P, P, P, P, P, S, MoERouteOpts, ctypes.POINTER(MoESavedActs), P, P,
                                          P, P, P, P, F, ctypes.c_int32, P, P, P, P, P, P, P, P, P, P, sz, P],
            "moe_layer_backward": [P, P, P, P, P, P, P, P, S, P, P, P, P, P, F, ctypes.c_int32, P, P, P, P, P, P, P,
                                   P, P, P, sz, P],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name in ("moe_workspace_size", "moe_permute_workspace_size", "moe_grouped_swiglu_workspace_size"):
            fn = getattr(L, name)
            fn.argtypes = [S]
            fn.restype = sz
        L.moe_backward_workspace_size.argtypes = [S, ctypes.c_int32]
        L.moe_backward_workspace_size.restype = sz
        L.moe_backward_logits_workspace_size.argtypes = [S, ctypes.c_int32, ctypes.c_int32]
        L.moe_backward_logits_workspace_size.restype = sz
        L.moe_fp8_scale_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
        L.moe_fp8_scale_bytes.restype = sz
        L.moe_fp8_tile_scale_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
        L.moe_fp8_tile_scale_bytes.restype = sz
        L.moe_ep_plan_size.argtypes = [ctypes.c_int32, S]
        L.moe_ep_plan_size.restype = sz
        L.moe_kernel_launch_count.argtypes = []
        L.moe_kernel_launch_count.restype = ctypes.c_uint64
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = ctypes.c_int
        _lib = L
    return _lib


def _p(t):
    """Device pointer of a tensor (None -> NULL; an int is taken as a pointer)."""
    if t is None:
        return None
    return t if isinstance(t, int) else t.data_ptr()


def _stream(stream, device=None):
    if stream is None:
        import torch
        return _handles()[1](torch.cuda.current_device() if device is None else device)
    return stream if isinstance(stream, int) else stream.cuda_stream


_bound: tuple = ()


def _handles():
    """The current device, and a device's current stream as a raw handle: torch's own short ways to them where it has
    these (a Stream object costs 3 us)."""
    global _bound
    if not _bound:
        import torch
        _bound = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                  getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream))
    return _bound


def _check(status: int, where: str):
    if status != 0:
        raise MoEError(status, where)


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


_tables: tuple = ()


def _prepare():
    """The dtypes by name and the entry points, as _call looks them up: one assignment, so that another thread finds
    both or neither."""
    global _tables
    import torch
    _tables = ({n: getattr(torch, n) for n in ("float32", "bfloat16", "int32", "uint8")},
               {n: getattr(lib(), n) for n in EXPORTS})
    return _tables


def _refuse(name, what, t, dtype, n):
    if t.dtype is not _tables[0][dtype]:
        raise MoEError(1, f"{name}: {what} must be {dtype}, got {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise MoEError(1, f"{name}: {what} must be contiguous with at least {n} elements, got {tuple(t.shape)}, strides "
                          f"{t.stride()}")
    raise MoEError(1, f"{name}: {what} must be on one CUDA device with the other tensors, got {t.device}")


def _call(name, stream, *args):
    """Call entry point ``name`` on the given arguments and the stream.  A tuple
    (argument name, tensor, dtype, elements) is checked before it is passed as
    a pointer: the dtype, a contiguous tensor of at least so many elements, on
    the device of the others.  None and raw pointers go through as they are.
    The call runs with the tensors' device current, on its current stream
    unless one is given."""
    dtypes, functions = _tables or _prepare()
    dev, out = -1, []
    for a in args:
        if type(a) is tuple:
            what, a, dtype, n = a
            if a is not None and type(a) is not int:
                d = a.get_device()
                if (d < 0 or dev != d and dev >= 0 or a.dtype is not dtypes[dtype] or a.numel() < n
                        or not a.is_contiguous()):
                    _refuse(name, what, a, dtype, n)
                dev = d
                a = a.data_ptr()
        out.append(a)
    fn = functions[name]
    if dev < 0:
        status = fn(*out, _stream(stream))
    else:
        device, raw_stream = _bound or _handles()
        if dev == device():
            status = fn(*out, raw_stream(dev) if stream is None else _stream(stream))
        else:
            import torch
            with torch.cuda.device(dev):
                status = fn(*out, _stream(stream, dev))
    if status:
        raise MoEError(status, name)


def _saved_ref(name, saved, shape, sets, device=-1):
    """Pointer to ``saved``, whose tensors of the expert sets ("" routed, "s"
    shared) hold the shape's rows, on the call's device."""
    if saved is None:
        return None
    room = getattr(saved, "room", None)
    if room:
        for pre in sets:
            need = shape.T * shape.k * shape.I if pre == "" else shape.T * shape.S * shape.Is
            if room[pre] is not None and room[pre] < need:
                raise MoEError(1, f"{name}: the saved {pre}a, {pre}g and their scales need {need} and {need // 32} bytes, "
                                  f"got {[saved.sizes.get(pre + n) for n in ('a', 'g', 'a_scale', 'g_scale')]}")
        if saved.device is not None and (saved.device < 0 or 0 <= device != saved.device):
            raise MoEError(1, f"{name}: saved activations must be on the CUDA device of the other tensors")
    return ctypes.byref(saved)


def _device(t) -> int:
    return -1 if t is None or isinstance(t, int) else t.get_device()


def _dt(shape) -> str:
    """dtype of x, the dense weights and the activations of a layer."""
    return "float32" if shape.dtype == MOE_F32 else "bfloat16"


# ---- entry points (same names and argument order as moe_gate.h) -----------

def moe_route(x, w_gate, bias, shape, topk_idx, topk_w, counts, affinity_out=None, stream=None):
    _check(lib().moe_route(_p(x), _p(w_gate), _p(bias), shape, _p(topk_idx), _p(topk_w), _p(counts),
                           _p(affinity_out), _stream(stream)), "moe_route")


def moe_load_and_bias_update(counts, shape, step, target, bias, load_out=None, stream=None):
    _check(lib().moe_load_and_bias_update(_p(counts), shape, ctypes.c_float(step), _p(target), _p(bias), _p(load_out),
                                          _stream(stream)), "moe_load_and_bias_update")


def moe_permute(x, topk_idx, counts, shape, x_perm, offsets, perm_tok, inv_row, workspace, stream=None):
    _check(lib().moe_permute(_p(x), _p(topk_idx), _p(counts), shape, _p(x_perm), _p(offsets), _p(perm_tok),
                             _p(inv_row), _p(workspace), _nbytes(workspace), _stream(stream)), "moe_permute")


def moe_permute_noalloc(x, topk_idx, counts, shape, x_perm, offsets, perm_tok, inv_row, stream=None):
    """moe_permute for callers that cannot provide scratch memory: the
    library uses a fixed array in its own device image instead (see
    moe_gate.h for the size limit and the sharing rules)."""
    _check(lib().moe_permute_noalloc(_p(x), _p(topk_idx), _p(counts), shape, _p(x_perm), _p(offsets), _p(perm_tok),
                                     _p(inv_row), _stream(stream)), "moe_permute_noalloc")


def moe_grouped_swiglu(x_perm, offsets, w1, w3, w2, x, ws1, ws3, ws2, shape, y_perm, shared_out, workspace,
                       stream=None):
    _check(lib().moe_grouped_swiglu(_p(x_perm), _p(offsets), _p(w1), _p(w3), _p(w2), _p(x), _p(ws1), _p(ws3),
                                    _p(ws2), shape, _p(y_perm), _p(shared_out), _p(workspace), _nbytes(workspace),
                                    _stream(stream)), "moe_grouped_swiglu")


def moe_expert_up(a, gather_idx, offsets, w1, w3, shape, expert_set, h, stream=None):
    _check(lib().moe_expert_up(_p(a), _p(gather_idx), _p(offsets), _p(w1), _p(w3), shape, expert_set, _p(h),
                               _stream(stream)), "moe_expert_up")


def moe_expert_down(h, offsets, w2, shape, expert_set, y, stream=None):
    _check(lib().moe_expert_down(_p(h), _p(offsets), _p(w2), shape, expert_set, _p(y), _stream(stream)),
           "moe_expert_down")


def moe_ffn_up(x_perm, offsets, w1, w3, x, ws1, ws3, shape, h, hs, stream=None):
    _check(lib().moe_ffn_up(_p(x_perm), _p(offsets), _p(w1), _p(w3), _p(x), _p(ws1), _p(ws3), shape, _p(h), _p(hs),
                            _stream(stream)), "moe_ffn_up")


def moe_ffn_down(h, offsets, w2, hs, ws2, shape, y_perm, shared_out, stream=None):
    _check(lib().moe_ffn_down(_p(h), _p(offsets), _p(w2), _p(hs), _p(ws2), shape, _p(y_perm), _p(shared_out),
                              _stream(stream)), "moe_ffn_down")


def moe_ffn_down_combine(h, offsets, w2, hs, ws2, perm_tok, topk_w, shape, y_acc, stream=None):
    _check(lib().moe_ffn_down_combine(_p(h), _p(offsets), _p(w2), _p(hs), _p(ws2), _p(perm_tok), _p(topk_w), shape,
                                      _p(y_acc), _stream(stream)), "moe_ffn_down_combine")


def moe_combine_finish(y_acc, shape, y, stream=None):
    _check(lib().moe_combine_finish(_p(y_acc), shape, _p(y), _stream(stream)), "moe_combine_finish")


def moe_combine(y_perm, topk_w, inv_row, shared_out, shape, y, stream=None):
    _check(lib().moe_combine(_p(y_perm), _p(topk_w), _p(inv_row), _p(shared_out), shape, _p(y), _stream(stream)),
           "moe_combine")


def moe_layer_forward(x, w_gate, bias, w1, w3, w2, ws1, ws3, ws2, shape, y, topk_idx, topk_w, counts, workspace,
                      stream=None):
    _check(lib().moe_layer_forward(_p(x), _p(w_gate), _p(bias), _p(w1), _p(w3), _p(w2), _p(ws1), _p(ws3), _p(ws2),
                                   shape, _p(y), _p(topk_idx), _p(topk_w), _p(counts), _p(workspace),
                                   _nbytes(workspace), _stream(stream)), "moe_layer_forward")


def moe_workspace_size(shape) -> int:
    return lib().moe_workspace_size(shape)


def moe_layer_backward(x, w_gate, w1, w3, w2, ws1, ws3, ws2, shape, topk_idx, topk_w, counts, affinity, dy, alpha,
                       seq_len, dx, dw_gate, dw1, dw3, dw2, dws1, dws3, dws2, balance_loss, workspace, stream=None):
    _check(lib().moe_layer_backward(_p(x), _p(w_gate), _p(w1), _p(w3), _p(w2), _p(ws1), _p(ws3), _p(ws2), shape,
                                    _p(topk_idx), _p(topk_w), _p(counts), _p(affinity), _p(dy), float(alpha),
                                    int(seq_len), _p(dx), _p(dw_gate), _p(dw1), _p(dw3), _p(dw2), _p(dws1), _p(dws3),
                                    _p(dws2), _p(balance_loss), _p(workspace), _nbytes(workspace), _stream(stream)),
           "moe_layer_backward")


def moe_backward_workspace_size(shape, seq_len: int = 0) -> int:
    return lib().moe_backward_workspace_size(shape, int(seq_len))


def moe_permute_workspace_size(shape) -> int:
    return lib().moe_permute_workspace_size(shape)


def moe_grouped_swiglu_workspace_size(shape) -> int:
    return lib().moe_grouped_swiglu_workspace_size(shape)


def moe_get_last_error(stream=None) -> int:
    return lib().moe_get_last_error(_stream(stream))


def moe_selftest_bounded_wait(limit_us: int, stream=None):
    _check(lib().moe_selftest_bounded_wait(limit_us, _stream(stream)), "moe_selftest_bounded_wait")


def moe_kernel_launch_count() -> int:
    return lib().moe_kernel_launch_count()


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def moe_abi_version() -> int:
    return lib().moe_abi_version()


# ---- FP8 experts -------------------------------------------------------------

MOE_SF_TOKENS, MOE_SF_WEIGHTS, MOE_SF_GATE, MOE_SF_UP = 0, 1, 2, 3


def moe_fp8_scale_bytes(rows, K, layout) -> int:
    return lib().moe_fp8_scale_bytes(rows, K, layout)


def moe_quantize_fp8(src, rows, kseg, nseg, layout, q, scales, stream=None):
    _check(lib().moe_quantize_fp8(_p(src), rows, kseg, nseg, layout, _p(q), _p(scales), _stream(stream)),
           "moe_quantize_fp8")


def fp8_scales(rows, K, layout, device):
    """An uninitialised device buffer for the tile scales of a [rows][K] matrix
    in the given layout (uint8, moe_fp8_scale_bytes long)."""
    import torch
    n = moe_fp8_scale_bytes(rows, K, layout)
    if n == 0:
        raise MoEError(1, "moe_fp8_scale_bytes: K must be a multiple of 128")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_fp8_tile_scale_bytes(rows, groups, K) -> int:
    return lib().moe_fp8_tile_scale_bytes(rows, groups, K)


def fp8_tile_images(rows, groups, K, device):
    """An uninitialised device buffer for the token tile images of `rows`
    operand rows in `groups` groups with K columns (uint8)."""
    import torch
    n = moe_fp8_tile_scale_bytes(rows, groups, K)
    if n == 0:
        raise MoEError(1, "moe_fp8_tile_scale_bytes: K must be a multiple of 128, 1 <= groups <= 256")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_fp8_tile_scales(src, src_rows, K, row_of, row_div, offsets, groups, rows, tiles, stream=None):
    _check(lib().moe_fp8_tile_scales(_p(src), src_rows, K, _p(row_of), row_div, _p(offsets), groups, rows, _p(tiles),
                                     _stream(stream)), "moe_fp8_tile_scales")


def moe_ffn_up_fp8(xq_perm, x_tiles, offsets, xq, xsh_tiles, experts, shape, h, hs, stream=None):
    _check(lib().moe_ffn_up_fp8(_p(xq_perm), _p(x_tiles), _p(offsets), _p(xq), _p(xsh_tiles), ctypes.byref(experts),
                                shape, _p(h), _p(hs), _stream(stream)), "moe_ffn_up_fp8")


def moe_ffn_up_fp8_quant(xq_perm, x_tiles, offsets, xq, xsh_tiles, experts, shape, hq, h_tiles, hsq, hs_tiles,
                         stream=None):
    _check(lib().moe_ffn_up_fp8_quant(_p(xq_perm), _p(x_tiles), _p(offsets), _p(xq), _p(xsh_tiles),
                                      ctypes.byref(experts), shape, _p(hq), _p(h_tiles), _p(hsq), _p(hs_tiles),
                                      _stream(stream)), "moe_ffn_up_fp8_quant")


def moe_ffn_down_fp8(hq, h_tiles, offsets, hsq, hs_tiles, experts, shape, y_perm, shared_out, stream=None):
    _check(lib().moe_ffn_down_fp8(_p(hq), _p(h_tiles), _p(offsets), _p(hsq), _p(hs_tiles), ctypes.byref(experts),
                                  shape, _p(y_perm), _p(shared_out), _stream(stream)), "moe_ffn_down_fp8")


def moe_layer_forward_fp8(x, w_gate, bias, experts, shape, y, topk_idx, topk_w, counts, workspace, stream=None):
    _check(lib().moe_layer_forward_fp8(_p(x), _p(w_gate), _p(bias), ctypes.byref(experts), shape, _p(y),
                                       _p(topk_idx), _p(topk_w), _p(counts), _p(workspace), _nbytes(workspace),
                                       _stream(stream)), "moe_layer_forward_fp8")


def quantize_experts_fp8(p: dict, stream=None) -> dict:
    """E4M3 copies of a layer's bf16 expert weights (device tensors) through
    moe_quantize_fp8: W1 and W3 (Ws1 and Ws3) with their scales in one gate/up
    buffer (MOE_SF_GATE, MOE_SF_UP), W2 in 128-row atoms (MOE_SF_WEIGHTS), the
    shared Ws2 [S][d][Is] as d rows across its S blocks.  Returns uint8 codes
    (the weights' own shapes) under w1q, w3q, w2q, ... and scale buffers under
    w13s, w2s, ws13s, ws2s."""
    import torch
    out = {}
    for a, b in (("w1", "w3"), ("ws1", "ws3")):
        w1, w3 = p.get(a), p.get(b)
        if w1 is None or w1.numel() == 0:
            continue
        rows, K = w1.numel() // w1.shape[-1], w1.shape[-1]
        sc = fp8_scales(rows, K, MOE_SF_GATE, w1.device)
        for n, w, lay in ((a, w1, MOE_SF_GATE), (b, w3, MOE_SF_UP)):
            q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
            moe_quantize_fp8(w, rows, K, 1, lay, q, sc, stream)
            out[n + "q"] = q
        out[a[:-1] + "13s"] = sc
    w = p["w2"]
    rows, K = w.numel() // w.shape[-1], w.shape[-1]
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    sc = fp8_scales(rows, K, MOE_SF_WEIGHTS, w.device)
    moe_quantize_fp8(w, rows, K, 1, MOE_SF_WEIGHTS, q, sc, stream)
    out["w2q"], out["w2s"] = q, sc
    w = p.get("ws2")
    if w is not None and w.numel() > 0:
        S, d, Is = w.shape
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        sc = fp8_scales(d, S * Is, MOE_SF_WEIGHTS, w.device)
        moe_quantize_fp8(w, d, Is, S, MOE_SF_WEIGHTS, q, sc, stream)
        out["ws2q"], out["ws2s"] = q, sc
    return out


# ---- routing from logits -----------------------------------------------------

def moe_gate_logits(x, w_gate, shape, logits, stream=None):
    T, d, E, dt = shape.T, shape.d, shape.E, _dt(shape)
    _call("moe_gate_logits", stream, ("x", x, dt, T * d), ("w_gate", w_gate, dt, E * d), shape,
          ("logits", logits, "float32", T * E))


def moe_route_logits(logits, bias, shape, opts, topk_idx, topk_w, counts, stream=None):
    T, E, k = shape.T, shape.E, shape.k
    _call("moe_route_logits", stream, ("logits", logits, "float32", T * E), ("bias", bias, "float32", E), shape, opts,
          ("topk_idx", topk_idx, "int32", T * k), ("topk_w", topk_w, "float32", T * k), ("counts", counts, "int32", E))


def moe_route_logits_backward(logits, topk_idx, dw, dscores, shape, opts, dlogits, stream=None):
    T, E, k = shape.T, shape.E, shape.k
    _call("moe_route_logits_backward", stream, ("logits", logits, "float32", T * E),
          ("topk_idx", topk_idx, "int32", T * k), ("dw", dw, "float32", T * k), ("dscores", dscores, "float32", T * E),
          shape, opts, ("dlogits", dlogits, "float32", T * E))


# ---- activations saved in 8 bits -----------------------------------------------

def saved_act_buffers(shape, device) -> dict:
    """Uninitialised device buffers for the saved pre-activations of a layer
    (uint8 tensors under MoESavedActs' field names; the shared ones only with
    shape.S > 0): pass saved_acts(...) of them to the calls."""
    import torch
    out = {}
    sets = [("", shape.T * shape.k, shape.I)] + ([("s", shape.T, shape.S * shape.Is)] if shape.S > 0 else [])
    for pre, rows, n in sets:
        for name in ("a", "g"):
            out[pre + name] = torch.empty((rows, n), dtype=torch.uint8, device=device)
            out[pre + name + "_scale"] = torch.empty(moe_fp8_scale_bytes(rows, n, MOE_SF_TOKENS), dtype=torch.uint8,
                                                     device=device)
    return out


def moe_ffn_up_save(x_perm, offsets, w1, w3, x, ws1, ws3, shape, h, hs, saved, stream=None):
    T, d, E, dt, SI = shape.T, shape.d, shape.E, _dt(shape), shape.S * shape.Is
    R, I = T * shape.k, shape.I
    _call("moe_ffn_up_save", stream, ("x_perm", x_perm, dt, R * d), ("offsets", offsets, "int32", E + 1),
          ("w1", w1, dt, E * I * d), ("w3", w3, dt, E * I * d), ("x", x, dt, T * d), ("ws1", ws1, dt, SI * d),
          ("ws3", ws3, dt, SI * d), shape, ("h", h, dt, R * I), ("hs", hs, dt, T * SI),
          _saved_ref("moe_ffn_up_save", saved, shape, ("",) if x is None or SI == 0 else ("", "s"), _device(x_perm)))


def moe_swiglu_backward_saved(saved, shape, expert_set, u, perm_tok, topk_w, dadg, h, dw, stream=None):
    R = shape.T * shape.k
    n = R * shape.I if expert_set == MOE_ROUTED else shape.T * shape.S * shape.Is
    ref = _saved_ref("moe_swiglu_backward_saved", saved, shape, ("",) if expert_set == MOE_ROUTED else ("s",), _device(u))
    _call("moe_swiglu_backward_saved", stream, ref, shape, expert_set, ("u", u, "float32", n),
          ("perm_tok", perm_tok, "int32", R), ("topk_w", topk_w, "float32", R), ("dadg", dadg, "bfloat16", 2 * n),
          ("h", h, "bfloat16", n), ("dw", dw, "float32", R))


# ---- the layer with routing from logits ------------------------------------------

def _layer_args(x, w_gate, w1, w3, w2, ws1, ws3, ws2, shape):
    """The checked weights of a layer, by name."""
    dt, d, SI = _dt(shape), shape.d, shape.S * shape.Is
    EId = shape.E * shape.I * d
    return dict(x=("x", x, dt, shape.T * d), w_gate=("w_gate", w_gate, dt, shape.E * d), w1=("w1", w1, dt, EId),
                w3=("w3", w3, dt, EId), w2=("w2", w2, dt, EId), ws1=("ws1", ws1, dt, SI * d),
                ws3=("ws3", ws3, dt, SI * d), ws2=("ws2", ws2, dt, SI * d))


def moe_layer_forward_logits(x, w_gate, bias, w1, w3, w2, ws1, ws3, ws2, shape, opts, y, logits, topk_idx, topk_w,
                             counts, saved, workspace, stream=None):
    T, E, k = shape.T, shape.E, shape.k
    a = _layer_args(x, w_gate, w1, w3, w2, ws1, ws3, ws2, shape)
    _call("moe_layer_forward_logits", stream, a["x"], a["w_gate"], ("bias", bias, "float32", E), a["w1"], a["w3"],
          a["w2"], a["ws1"], a["ws3"], a["ws2"], shape, opts, ("y", y, _dt(shape), T * shape.d),
          ("logits", logits, "float32", T * E), ("topk_idx", topk_idx, "int32", T * k),
          ("topk_w", topk_w, "float32", T * k), ("counts", counts, "int32", E),
          _saved_ref("moe_layer_forward_logits", saved, shape, ("", "s") if shape.S > 0 else ("",), _device(x)),
          ("workspace", workspace, "uint8", 0), _nbytes(workspace))


def moe_backward_logits_workspace_size(shape, seq_len: int = 0, saved: bool = False) -> int:
    return lib().moe_backward_logits_workspace_size(shape, int(seq_len), int(bool(saved)))


def moe_layer_backward_logits(x, w_gate, w1, w3, w2, ws1, ws3, ws2, shape, opts, saved, logits, topk_idx, topk_w,
                              counts, dscores, dy, alpha, seq_len, dx, dw_gate, dw1, dw3, dw2, dws1, dws3, dws2,
                              balance_loss, workspace, stream=None):
    T, d, E, k, SI = shape.T, shape.d, shape.E, shape.k, shape.S * shape.Is
    EId = E * shape.I * d
    f = lambda name, t, n: (name, t, "float32", n)
    a = _layer_args(x, w_gate, w1, w3, w2, ws1, ws3, ws2, shape)
    _call("moe_layer_backward_logits", stream, a["x"], a["w_gate"], a["w1"], a["w3"], a["w2"], a["ws1"], a["ws3"],
          a["ws2"], shape, opts,
          _saved_ref("moe_layer_backward_logits", saved, shape, ("", "s") if shape.S > 0 else ("",), _device(x)),
          f("logits", logits, T * E), ("topk_idx", topk_idx, "int32", T * k),
          f("topk_w", topk_w, T * k), ("counts", counts, "int32", E), f("dscores", dscores, T * E), f("dy", dy, T * d),
          float(alpha), int(seq_len), f("dx", dx, T * d), f("dw_gate", dw_gate, E * d), f("dw1", dw1, EId),
          f("dw3", dw3, EId), f("dw2", dw2, EId), f("dws1", dws1, SI * d), f("dws3", dws3, SI * d),
          f("dws2", dws2, SI * d), f("balance_loss", balance_loss, 1), ("workspace", workspace, "uint8", 0),
          _nbytes(workspace))


# ---- expert parallelism --------------------------------------------------------

def _ptr_array(bufs):
    arr = (ctypes.c_void_p * len(bufs))()
    for i, b in enumerate(bufs):
        arr[i] = b if isinstance(b, int) else b.data_ptr()
    return arr


def moe_ep_plan_size(world, shape) -> int:
    return lib().moe_ep_plan_size(world, shape)


def moe_ep_plan(counts_all, world, rank, shape, recv_capacity, plan, recv_offsets, stream=None):
    _check(lib().moe_ep_plan(_p(counts_all), world, rank, shape, recv_capacity, _p(plan), _p(recv_offsets),
                             _stream(stream)),
           "moe_ep_plan")


def moe_ep_dispatch(x, perm_tok, plan, world, rank, shape, recv_bufs, stream=None):
    """recv_bufs: per rank, its receive buffer (tensor or device pointer valid here)."""
    _check(lib().moe_ep_dispatch(_p(x), _p(perm_tok), _p(plan), world, rank, shape, _ptr_array(recv_bufs),
                                 _stream(stream)), "moe_ep_dispatch")


def moe_ep_return(y_recv, plan, world, rank, shape, back_bufs, stream=None):
    """back_bufs: per rank, its return buffer (tensor or device pointer valid here)."""
    _check(lib().moe_ep_return(_p(y_recv), _p(plan), world, rank, shape, _ptr_array(back_bufs), _stream(stream)),
           "moe_ep_return")
