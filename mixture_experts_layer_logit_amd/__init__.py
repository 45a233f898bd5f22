"""MI355X (gfx950) MoE-layer forward: Python binding of libmoe.so.

The binding only marshals arguments: every step of the layer runs in the HIP
kernels behind the C ABI of ``include/moe.h``.  Torch tensors provide device
memory and the current HIP stream; there is no CPU or PyTorch fallback, and
loading fails loudly when the library has not been built.

Entry points (same names as the C ABI): moe_capacity, moe_workspace_size,
moe_route, moe_permute, moe_expert_up, moe_expert_down, moe_grouped_ffn,
moe_combine, moe_forward, moe_router_stats, moe_shared_workspace_size,
moe_shared_expert, moe_combine_shared, moe_quantize_fp8, moe_fp8_workspace_size,
moe_expert_up_fp8, moe_expert_down_fp8, moe_forward_fp8, moe_forward_train,
moe_backward_workspace_size, moe_backward, moe_forward_noalloc,
moe_quantize_fp8_block, moe_fp8_block_workspace_size, moe_expert_up_fp8_block,
moe_expert_down_fp8_block, moe_forward_fp8_block, moe_balance_workspace_size,
moe_balance_loss.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_LIB names another build of the same sources (the host-sanitizer build)
LIB_PATH = os.environ.get("MOE_LIB") or os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_ACT_RELU, MOE_ACT_SWIGLU = 0, 1
MOE_F32, MOE_BF16 = 0, 1
MOE_SCALE_E8M0, MOE_SCALE_F32 = 0, 1

EXPORTS = ("moe_status_string", "moe_last_error", "moe_capacity", "moe_workspace_size", "moe_route",
           "moe_permute", "moe_expert_up", "moe_expert_down", "moe_grouped_ffn", "moe_combine", "moe_forward",
           "moe_router_stats", "moe_shared_workspace_size", "moe_shared_expert", "moe_combine_shared",
           "moe_quantize_fp8", "moe_fp8_workspace_size", "moe_expert_up_fp8", "moe_expert_down_fp8",
           "moe_forward_fp8", "moe_forward_train", "moe_backward_workspace_size", "moe_backward",
           "moe_forward_noalloc", "moe_quantize_fp8_block", "moe_fp8_block_workspace_size",
           "moe_expert_up_fp8_block", "moe_expert_down_fp8_block", "moe_forward_fp8_block",
           "moe_balance_workspace_size", "moe_balance_loss")


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("F", ctypes.c_int32), ("act", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("normalize", ctypes.c_int32), ("lambda_", ctypes.c_float), ("capacity_factor", ctypes.c_float)]


class RouteInfo(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("slot", ctypes.c_void_p), ("src_token", ctypes.c_void_p)]


class RouterLosses(ctypes.Structure):
    _fields_ = [("aux_coef", ctypes.c_float), ("z_coef", ctypes.c_float)]


class Saved(ctypes.Structure):
    _fields_ = [("u", ctypes.c_void_p), ("h", ctypes.c_void_p), ("y_perm", ctypes.c_void_p)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libmoe.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run python -m mixture_experts_layer_logit_amd.build")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    PP = ctypes.POINTER(Problem)
    st = ctypes.c_int
    lib.moe_status_string.argtypes = [st]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_last_error.argtypes = []
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_capacity.argtypes = [PP, ctypes.POINTER(ctypes.c_int32)]
    lib.moe_workspace_size.argtypes = [PP, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_route.argtypes = [PP, P, P, P, P, P, P, P]
    lib.moe_permute.argtypes = [PP, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_expert_up.argtypes = [PP, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_expert_down.argtypes = [PP, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_grouped_ffn.argtypes = [PP, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_combine.argtypes = [PP, P, P, P, P, P]
    lib.moe_forward.argtypes = [PP, P, P, P, P, P, P, P, ctypes.POINTER(RouteInfo), P, ctypes.c_size_t, P]
    lib.moe_forward_noalloc.argtypes = [PP, P, P, P, P, P, P, P, ctypes.POINTER(RouteInfo), P]
    lib.moe_router_stats.argtypes = [PP, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_shared_workspace_size.argtypes = [PP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_shared_expert.argtypes = [PP, ctypes.c_int32, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_combine_shared.argtypes = [PP, P, P, P, P, P, P]
    lib.moe_quantize_fp8.argtypes = [P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, P, P, P]
    lib.moe_fp8_workspace_size.argtypes = [PP, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_expert_up_fp8.argtypes = [PP, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_expert_down_fp8.argtypes = [PP, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_forward_fp8.argtypes = [PP, P, P, P, P, P, P, P, P, P, ctypes.POINTER(RouteInfo), P, ctypes.c_size_t,
                                    P]
    lib.moe_forward_train.argtypes = [PP, P, P, P, P, P, P, P, ctypes.POINTER(RouteInfo), ctypes.POINTER(Saved), P,
                                      ctypes.c_size_t, P]
    lib.moe_backward_workspace_size.argtypes = [PP, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_backward.argtypes = [PP, P, P, P, P, P, P, ctypes.POINTER(RouteInfo), ctypes.POINTER(Saved),
                                 ctypes.POINTER(RouterLosses), P, P, P, P, P, P, ctypes.c_size_t, P]
    i32, size = ctypes.c_int32, ctypes.c_size_t
    lib.moe_quantize_fp8_block.argtypes = [P, i32, ctypes.c_int64, i32, i32, P, P, i32, P]
    lib.moe_fp8_block_workspace_size.argtypes = [PP, ctypes.POINTER(size)]
    lib.moe_expert_up_fp8_block.argtypes = [PP, P, P, P, P, P, P, i32, P, P, P, size, P]
    lib.moe_expert_down_fp8_block.argtypes = [PP, P, P, P, P, P, i32, P, P, size, P]
    lib.moe_forward_fp8_block.argtypes = [PP, P, P, P, P, P, P, P, i32, P, P, ctypes.POINTER(RouteInfo), P, size, P]
    lib.moe_balance_workspace_size.argtypes = [PP, i32, ctypes.POINTER(size)]
    lib.moe_balance_loss.argtypes = [PP, P, P, P, i32, ctypes.c_float, ctypes.c_float, P, P, P, P, size, P]
    for name in EXPORTS[2:]:
        getattr(lib, name).restype = st
    _lib = lib
    return lib


def status_name(status: int) -> str:
    try:
        return load().moe_status_string(status).decode()
    except ImportError:
        return str(status)


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, load().moe_last_error().decode())


def problem(T, d, E, k, F, act="relu", dtype="bf16", normalize=False, lam=1.0, cf=0.0) -> Problem:
    """Build the moe_problem struct (act: "relu"|"swiglu", dtype: "f32"|"bf16")."""
    a = {"relu": MOE_ACT_RELU, "swiglu": MOE_ACT_SWIGLU}.get(act, act)
    t = {"f32": MOE_F32, "bf16": MOE_BF16}.get(dtype, dtype)
    return Problem(int(T), int(d), int(E), int(k), int(F), int(a), int(t), int(bool(normalize)), float(lam),
                   float(cf))


def _ptr(t):
    """Device address of a tensor (None -> NULL); plain ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


_current_stream = None


def _stream(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch
            torch.cuda.init()
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", None)
            # the stream's handle without a Stream object around it, which takes
            # longer to make than a small kernel to launch
            _current_stream = (lambda: raw(device())) if raw and device else (
                lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_capacity(p: Problem) -> int:
    c = ctypes.c_int32()
    _check(load().moe_capacity(ctypes.byref(p), ctypes.byref(c)))
    return c.value


def moe_workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def _nbytes(ws):
    if ws is None:
        return 0
    return ws.numel() * ws.element_size()


def moe_route(p, x, Wg, bg, logits, topk_idx, topk_w, stream=None):
    _check(load().moe_route(ctypes.byref(p), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(logits), _ptr(topk_idx),
                            _ptr(topk_w), _stream(stream)))


def moe_permute(p, topk_idx, x, counts, offsets, slot, src_token, x_perm, ws, stream=None):
    _check(load().moe_permute(ctypes.byref(p), _ptr(topk_idx), _ptr(x), _ptr(counts), _ptr(offsets), _ptr(slot),
                              _ptr(src_token), _ptr(x_perm), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_expert_up(p, a, src_token, offsets, W1, h, ws=None, stream=None):
    """a is x_perm (src_token None) or x (rows gathered through src_token)."""
    _check(load().moe_expert_up(ctypes.byref(p), _ptr(a), _ptr(src_token), _ptr(offsets), _ptr(W1), _ptr(h),
                                _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_expert_down(p, h, offsets, W2, y_perm, ws=None, stream=None):
    _check(load().moe_expert_down(ctypes.byref(p), _ptr(h), _ptr(offsets), _ptr(W2), _ptr(y_perm), _ptr(ws),
                                  _nbytes(ws), _stream(stream)))


def moe_grouped_ffn(p, x_perm, offsets, W1, W2, y_perm, ws, stream=None):
    _check(load().moe_grouped_ffn(ctypes.byref(p), _ptr(x_perm), _ptr(offsets), _ptr(W1), _ptr(W2), _ptr(y_perm),
                                  _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_combine(p, y_perm, slot, topk_w, y, stream=None):
    _check(load().moe_combine(ctypes.byref(p), _ptr(y_perm), _ptr(slot), _ptr(topk_w), _ptr(y), _stream(stream)))


def moe_forward(p, x, Wg, bg, W1, W2, y, logits=None, info=None, ws=None, stream=None):
    """info: optional dict with any of topk_idx, topk_w, counts, offsets, slot, src_token tensors."""
    ri = None
    if info:
        ri = RouteInfo(*[_ptr(info.get(f)) for f, _ in RouteInfo._fields_])
    _check(load().moe_forward(ctypes.byref(p), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1), _ptr(W2), _ptr(y),
                              _ptr(logits), ctypes.byref(ri) if ri is not None else None, _ptr(ws), _nbytes(ws),
                              _stream(stream)))


def moe_forward_noalloc(p, x, Wg, bg, W1, W2, y, logits=None, info=None, stream=None):
    """moe_forward with the library's own device scratch as workspace (no
    allocation; problems up to 32 MiB of workspace)."""
    ri = None
    if info:
        ri = RouteInfo(*[_ptr(info.get(f)) for f, _ in RouteInfo._fields_])
    _check(load().moe_forward_noalloc(ctypes.byref(p), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1), _ptr(W2), _ptr(y),
                                      _ptr(logits), ctypes.byref(ri) if ri is not None else None, _stream(stream)))


def moe_router_stats(p, logits, counts, offsets, frac, mean_prob, scalars, ws, stream=None):
    """scalars [3] = (aux loss without coefficient, Z-loss, drop rate)."""
    _check(load().moe_router_stats(ctypes.byref(p), _ptr(logits), _ptr(counts), _ptr(offsets), _ptr(frac),
                                   _ptr(mean_prob), _ptr(scalars), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_shared_workspace_size(p, Fs) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_shared_workspace_size(ctypes.byref(p), int(Fs), ctypes.byref(n)))
    return n.value


def moe_shared_expert(p, Fs, x, Ws1, Ws2, y_shared, ws, stream=None):
    _check(load().moe_shared_expert(ctypes.byref(p), int(Fs), _ptr(x), _ptr(Ws1), _ptr(Ws2), _ptr(y_shared),
                                    _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_combine_shared(p, y_perm, slot, topk_w, y_shared, y, stream=None):
    _check(load().moe_combine_shared(ctypes.byref(p), _ptr(y_perm), _ptr(slot), _ptr(topk_w), _ptr(y_shared),
                                     _ptr(y), _stream(stream)))


def moe_quantize_fp8(src, codes, scales, stream=None):
    """Rows of src (fp32 or bf16 tensor [rows, K]) to E4M3 codes (uint8 [rows, K])
    and power-of-two row scales (fp32 [rows])."""
    import torch
    dt = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}[src.dtype]
    rows, K = src.shape[0], src.numel() // max(src.shape[0], 1)
    _check(load().moe_quantize_fp8(_ptr(src), dt, rows, K, _ptr(codes), _ptr(scales), _stream(stream)))


def moe_fp8_workspace_size(p) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_fp8_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def moe_expert_up_fp8(p, aq, a_scale, src_token, offsets, W1q, w1s, h, ws=None, stream=None):
    _check(load().moe_expert_up_fp8(ctypes.byref(p), _ptr(aq), _ptr(a_scale), _ptr(src_token), _ptr(offsets),
                                    _ptr(W1q), _ptr(w1s), _ptr(h), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_expert_down_fp8(p, hq, hs, offsets, W2q, w2s, y_perm, ws=None, stream=None):
    _check(load().moe_expert_down_fp8(ctypes.byref(p), _ptr(hq), _ptr(hs), _ptr(offsets), _ptr(W2q), _ptr(w2s),
                                      _ptr(y_perm), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_forward_fp8(p, x, Wg, bg, W1q, w1s, W2q, w2s, y, logits=None, info=None, ws=None, stream=None):
    ri = None
    if info:
        ri = RouteInfo(*[_ptr(info.get(f)) for f, _ in RouteInfo._fields_])
    _check(load().moe_forward_fp8(ctypes.byref(p), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1q), _ptr(w1s), _ptr(W2q),
                                  _ptr(w2s), _ptr(y), _ptr(logits), ctypes.byref(ri) if ri is not None else None,
                                  _ptr(ws), _nbytes(ws), _stream(stream)))


def _route_info(info):
    return RouteInfo(*[_ptr(info.get(f)) for f, _ in RouteInfo._fields_])


def _saved(saved):
    return Saved(*[_ptr(saved.get(f)) for f, _ in Saved._fields_])


def moe_forward_train(p, x, Wg, bg, W1, W2, y, logits, info, saved, ws=None, stream=None):
    """info: dict of every route-info tensor; saved: dict of u, h, y_perm tensors."""
    ri, sv = _route_info(info), _saved(saved)
    _check(load().moe_forward_train(ctypes.byref(p), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1), _ptr(W2), _ptr(y),
                                    _ptr(logits), ctypes.byref(ri), ctypes.byref(sv), _ptr(ws), _nbytes(ws),
                                    _stream(stream)))


def moe_backward_workspace_size(p) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_backward_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def moe_backward(p, dy, x, Wg, W1, W2, logits, info, saved, dx, dWg, dbg, dW1, dW2, ws=None, stream=None,
                 aux_coef=0.0, z_coef=0.0):
    """aux_coef, z_coef: coefficients of the balancing losses (auxiliary
    loss, Z-loss) whose gradients are added; both 0 passes no losses."""
    ri = _route_info(info) if info is not None else None
    sv = _saved(saved) if saved is not None else None
    ls = RouterLosses(float(aux_coef), float(z_coef)) if (aux_coef or z_coef) else None
    _check(load().moe_backward(ctypes.byref(p), _ptr(dy), _ptr(x), _ptr(Wg), _ptr(W1), _ptr(W2), _ptr(logits),
                               ctypes.byref(ri) if ri is not None else None,
                               ctypes.byref(sv) if sv is not None else None,
                               ctypes.byref(ls) if ls is not None else None, _ptr(dx), _ptr(dWg), _ptr(dbg),
                               _ptr(dW1), _ptr(dW2), _ptr(ws), _nbytes(ws), _stream(stream)))


_scale_types, _src_types = {}, {}
_f32 = _i32 = _bf16 = _codes = None
_INFO = tuple(f for f, _ in RouteInfo._fields_)


def _fill_types():
    import torch
    global _f32, _i32, _bf16, _codes
    _f32, _i32, _bf16 = torch.float32, torch.int32, torch.bfloat16
    _codes = (torch.uint8, torch.float8_e4m3fn, torch.int8)
    _scale_types.update({torch.float32: MOE_SCALE_F32, torch.uint8: MOE_SCALE_E8M0,
                         torch.float8_e8m0fnu: MOE_SCALE_E8M0})
    _src_types.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16})


def _refuse(types, sizes=()):
    """TypeError for the first (name, tensor, type or types) whose tensor has another
    element type, ValueError for the first (name, tensor, least) with fewer elements:
    the kernels would read the bytes as something else, or go past their end.  None
    and plain addresses pass."""
    for name, t, kind in types:
        if t is None or isinstance(t, int):
            continue
        if (t.dtype not in kind) if kind is _codes else (t.dtype is not kind):
            raise TypeError(f"{name}: {' or '.join(map(str, kind[:2])) if kind is _codes else kind}, not {t.dtype}")
    for name, t, least in sizes:
        if t is not None and not isinstance(t, int) and t.numel() < least:
            raise ValueError(f"{name}: {t.numel()} elements, {least} are needed")


def _scale_type(scales) -> int:
    """MOE_SCALE_* of a tensor of block scales, by its element type."""
    if _f32 is None:
        _fill_types()
    kind = _scale_types.get(scales.dtype)
    if kind is None:
        raise TypeError(f"block scales are float32 or E8M0 (uint8 or float8_e8m0fnu), not {scales.dtype}")
    return kind


def _e8m0(scales, name):
    if scales is not None and not isinstance(scales, int) and _scale_type(scales) != MOE_SCALE_E8M0:
        raise TypeError(f"{name}: activation scales are E8M0 (uint8 or float8_e8m0fnu), not {scales.dtype}")
    return scales


def moe_quantize_fp8_block(src, codes, scales, block_rows=1, stream=None):
    """Rows of src (fp32 or bf16 tensor [rows, K]) to E4M3 codes (uint8 [rows, K])
    with a power-of-two scale per block of block_rows (1 or 128) x 128 values;
    scales [ceil(rows / block_rows), K / 128] is uint8 / float8_e8m0fnu (E8M0) or fp32.
    Here and below codes may also be float8_e4m3fn; other types raise TypeError,
    outputs with too few elements ValueError."""
    kind = _scale_type(scales)
    dt = _src_types.get(src.dtype)
    if dt is None:
        raise TypeError(f"src is float32 or bfloat16, not {src.dtype}")
    n, K = src.numel(), src.shape[-1]
    rows = n // (K or 1)
    least = (rows if block_rows <= 1 else -(-rows // block_rows)) * (K // 128)
    try:  # as in moe_balance_loss
        fits = codes.dtype in _codes and codes.numel() >= n and scales.numel() >= least
    except AttributeError:
        fits = False
    if not fits:
        _refuse((("codes", codes, _codes),), (("codes", codes, n), ("scales", scales, least)))
    _check(load().moe_quantize_fp8_block(_ptr(src), dt, rows, K, int(block_rows), _ptr(codes), _ptr(scales), kind,
                                         _stream(stream)))


def moe_fp8_block_workspace_size(p) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_fp8_block_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def moe_expert_up_fp8_block(p, aq, a_scale, src_token, offsets, W1q, w1s, hq, hs, ws=None, stream=None):
    """aq, a_scale: codes and E8M0 scales of x (rows gathered through src_token) or
    of the permuted rows (src_token None); w1s: E8M0 or fp32 scales; hq, hs: out."""
    kind = _scale_type(w1s)
    _refuse((("aq", aq, _codes), ("src_token", src_token, _i32), ("offsets", offsets, _i32), ("W1q", W1q, _codes),
             ("hq", hq, _codes)))
    _check(load().moe_expert_up_fp8_block(ctypes.byref(p), _ptr(aq), _ptr(_e8m0(a_scale, "a_scale")),
                                          _ptr(src_token), _ptr(offsets), _ptr(W1q), _ptr(w1s), kind,
                                          _ptr(hq), _ptr(_e8m0(hs, "hs")), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_expert_down_fp8_block(p, hq, hs, offsets, W2q, w2s, y_perm, ws=None, stream=None):
    kind = _scale_type(w2s)
    _refuse((("hq", hq, _codes), ("offsets", offsets, _i32), ("W2q", W2q, _codes), ("y_perm", y_perm, _bf16)))
    _check(load().moe_expert_down_fp8_block(ctypes.byref(p), _ptr(hq), _ptr(_e8m0(hs, "hs")), _ptr(offsets),
                                            _ptr(W2q), _ptr(w2s), kind, _ptr(y_perm), _ptr(ws),
                                            _nbytes(ws), _stream(stream)))


def moe_forward_fp8_block(p, x, Wg, bg, W1q, w1s, W2q, w2s, y, logits=None, info=None, ws=None, stream=None):
    """The layer with block-scaled FP8 experts; w1s and w2s of one type (E8M0 or fp32)."""
    kind = _scale_type(w1s)
    if _scale_type(w2s) != kind:
        raise TypeError("w1s and w2s must be scales of one type")
    T, E = p.T, p.E
    n = T * p.d
    try:  # as in moe_balance_loss: the loops over names take 4 us
        fits = (x.dtype is _bf16 and y.dtype is _bf16 and W1q.dtype in _codes and W2q.dtype in _codes
                and (Wg is None or Wg.dtype is _bf16) and (bg is None or bg.dtype is _f32)
                and (logits is None or logits.dtype is _f32 and logits.numel() >= T * E)
                and x.numel() >= n and y.numel() >= n)
    except AttributeError:
        fits = False
    if not fits:
        _refuse((("x", x, _bf16), ("Wg", Wg, _bf16), ("bg", bg, _f32), ("W1q", W1q, _codes), ("W2q", W2q, _codes),
                 ("y", y, _bf16), ("logits", logits, _f32)), (("x", x, n), ("y", y, n), ("logits", logits, T * E)))
    if info:
        least, choices = {"counts": E, "offsets": E + 1}, T * p.k
        for f in _INFO:
            t = info.get(f)
            if t is not None and not isinstance(t, int):
                of, n = _f32 if f == "topk_w" else _i32, least.get(f, choices)
                if t.dtype is not of or t.numel() < n:
                    _refuse(((f, t, of),), ((f, t, n),))
    ri = _route_info(info) if info else None
    _check(load().moe_forward_fp8_block(ctypes.byref(p), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1q), _ptr(w1s),
                                        _ptr(W2q), _ptr(w2s), kind, _ptr(y), _ptr(logits),
                                        ctypes.byref(ri) if ri is not None else None, _ptr(ws), _nbytes(ws),
                                        _stream(stream)))


def moe_balance_workspace_size(p, n_seq) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_balance_workspace_size(ctypes.byref(p), int(n_seq), ctypes.byref(n)))
    return n.value


def moe_balance_loss(p, logits, topk_idx, seq_offsets, counts, losses, dlogits, aux_coef=0.0, z_coef=0.0, ws=None,
                     stream=None):
    """counts [n_seq, E] int32, losses [2] = (aux, Z), dlogits [T, E] (or None) of
    the sequences seq_offsets [n_seq + 1] int32 (None: one sequence of all tokens).
    logits [T, E], losses and dlogits are float32, topk_idx [T, k] int32: other types
    raise TypeError, tensors with too few elements ValueError."""
    if _f32 is None:
        _fill_types()
    n_seq, E, T = 1 if seq_offsets is None else seq_offsets.numel() - 1, p.E, p.T
    cells = T * E
    try:  # in one expression: a small call takes 6 us, the loops over names 2 of them
        fits = (logits.dtype is _f32 and topk_idx.dtype is _i32 and counts.dtype is _i32 and losses.dtype is _f32
                and (seq_offsets is None or seq_offsets.dtype is _i32)
                and (dlogits is None or dlogits.dtype is _f32 and dlogits.numel() >= cells)
                and logits.numel() >= cells and topk_idx.numel() >= T * p.k and counts.numel() >= n_seq * E
                and losses.numel() >= 2)
    except AttributeError:  # None or a plain address among them
        fits = False
    if not fits:
        _refuse((("logits", logits, _f32), ("topk_idx", topk_idx, _i32), ("seq_offsets", seq_offsets, _i32),
                 ("counts", counts, _i32), ("losses", losses, _f32), ("dlogits", dlogits, _f32)),
                (("logits", logits, cells), ("topk_idx", topk_idx, T * p.k), ("counts", counts, n_seq * E),
                 ("losses", losses, 2), ("dlogits", dlogits, cells)))
    _check(load().moe_balance_loss(ctypes.byref(p), _ptr(logits), _ptr(topk_idx), _ptr(seq_offsets), n_seq,
                                   float(aux_coef), float(z_coef), _ptr(counts), _ptr(losses), _ptr(dlogits),
                                   _ptr(ws), _nbytes(ws), _stream(stream)))
