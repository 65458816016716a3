"""ctypes binding of libmoe_mi355x.so: argument marshalling only.

Each function takes torch device tensors (or None), passes their data pointers and the current
HIP stream to the C entry point of the same name (include/moe.h) and raises MoEError on a
non-zero status. No computation happens here. If the library has not been built the first
call raises; there is no fallback path.
"""
import ctypes
import functools
import os
import re

import torch

from .configs import LayerConfig

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_MXFP4, MOE_INT8 = 0, 1, 2, 3, 4
MOE_SOFTMAX, MOE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2_SUM = 0, 1
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_HIP", 5: "MOE_ERR_DEVICE"}


class MoEError(RuntimeError):
    def __init__(self, status, where, detail):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("K", ctypes.c_int32), ("score_fn", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("route_scale", ctypes.c_float),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("I_shared", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class MoeNormConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("quant", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("residual_out_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64)]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_SIGS = {
    "moe_check_config": (_I, [_P]),
    "moe_workspace_size": (ctypes.c_size_t, [_P]),
    "moe_route": (_I, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_route_logits": (_I, [_P, _P, _P, _P, _P, _P]),
    "moe_update_bias": (_I, [_I, _P, _P, ctypes.c_float, _P]),
    "moe_permute": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_permute_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_expert_ffn": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn_gather": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                   _P]),
    "moe_combine": (_I, [_P, _P, _P, _P, _P, _P, _P]),
    "moe_layer_decode": (_I, [_P] + [_P] * 21 + [ctypes.c_size_t, _P]),
    "moe_quantize_fp8": (_I, [_I, _I, _P, _P, _P, _P]),
    "moe_quantize_mx": (_I, [_I, _I, _P, _P, _P, _P]),
    "moe_quantize_int8": (_I, [_I, _I, _P, _P, _P, _P]),
    "moe_rmsnorm": (_I, [_P] * 9),
    "moe_gemm_int8_workspace_size": (ctypes.c_size_t, []),
    "moe_gemm_int8": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, ctypes.c_size_t, _P]),
    "moe_get_device_error": (_I, [_P, ctypes.POINTER(_I), _P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_profile_enable": (None, [_I]),
    "moe_profile_reset": (None, []),
    "moe_profile_read": (_I, [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                              ctypes.POINTER(_I), _I]),
}

_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_layer_07_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions():
    """Names of the functions include/moe.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(moe_\w+)\s*\(", text, re.M)))


def make_config(cfg: LayerConfig) -> MoeConfig:
    dt = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8": MOE_FP8_E4M3, "mxfp4": MOE_MXFP4, "int8": MOE_INT8}[cfg.dtype]
    return MoeConfig(cfg.T, cfg.H, cfg.I, cfg.E, cfg.K,
                     MOE_SOFTMAX if cfg.score == "softmax" else MOE_SIGMOID,
                     1 if cfg.renorm else 0, float(cfg.route_scale), cfg.n_group,
                     cfg.topk_group if cfg.n_group > 1 else 1,
                     MOE_GROUP_TOP2_SUM if cfg.group_rule == "top2_sum" else MOE_GROUP_MAX,
                     dt, cfg.I_shared, MOE_F32 if cfg.out == "f32" else MOE_BF16)


def _cfg(cfg):
    c = cfg if isinstance(cfg, MoeConfig) else make_config(cfg)
    return c, ctypes.byref(c)


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # (the raw handle: a Stream object costs 2.5 us per call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(status, where):
    if status != 0:
        raise MoEError(status, where, lib().moe_last_error().decode())


def moe_check_config(cfg):
    c, pc = _cfg(cfg)
    _check(lib().moe_check_config(pc), "moe_check_config")


def moe_workspace_size(cfg) -> int:
    c, pc = _cfg(cfg)
    return int(lib().moe_workspace_size(pc))


def moe_route(cfg, x, w_router, bias, topk_ids, topk_weights, ws, stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_route(pc, _p(x), _p(w_router), _p(bias), _p(topk_ids), _p(topk_weights),
                           _p(ws), ws.numel() * ws.element_size(), _stream(stream)), "moe_route")


def moe_route_logits(cfg, logits, bias, topk_ids, topk_weights, stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_route_logits(pc, _p(logits), _p(bias), _p(topk_ids), _p(topk_weights),
                                  _stream(stream)), "moe_route_logits")


def moe_update_bias(n_experts, counts, bias, gamma, stream=None):
    _check(lib().moe_update_bias(int(n_experts), _p(counts), _p(bias), float(gamma), _stream(stream)),
           "moe_update_bias")


def moe_permute(cfg, topk_ids, counts, offsets, sorted_pair, pair_pos, x, x_perm, x_perm_scale, ws,
                stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_permute(pc, _p(topk_ids), _p(counts), _p(offsets), _p(sorted_pair),
                             _p(pair_pos), _p(x), _p(x_perm), _p(x_perm_scale), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "moe_permute")


def moe_permute_noalloc(cfg, topk_ids, counts, offsets, sorted_pair, pair_pos, x, x_perm, x_perm_scale,
                        stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_permute_noalloc(pc, _p(topk_ids), _p(counts), _p(offsets), _p(sorted_pair),
                                     _p(pair_pos), _p(x), _p(x_perm), _p(x_perm_scale), _stream(stream)),
           "moe_permute_noalloc")


def moe_expert_ffn(cfg, n_experts, n_rows, inter, offsets, x_rows, x_scale, w13, w13_scale, w2,
                   w2_scale, y_rows, ws, stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_expert_ffn(pc, n_experts, n_rows, inter, _p(offsets), _p(x_rows), _p(x_scale),
                                _p(w13), _p(w13_scale), _p(w2), _p(w2_scale), _p(y_rows), _p(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "moe_expert_ffn")


def moe_expert_ffn_gather(cfg, n_experts, n_rows, inter, offsets, sorted_pair, x, x_scale, w13,
                          w13_scale, w2, w2_scale, y_rows, ws, stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_expert_ffn_gather(pc, n_experts, n_rows, inter, _p(offsets), _p(sorted_pair), _p(x),
                                       _p(x_scale), _p(w13), _p(w13_scale), _p(w2), _p(w2_scale),
                                       _p(y_rows), _p(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)), "moe_expert_ffn_gather")


def moe_combine(cfg, pair_pos, topk_weights, y_perm, y_shared, out, stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_combine(pc, _p(pair_pos), _p(topk_weights), _p(y_perm), _p(y_shared), _p(out),
                             _stream(stream)), "moe_combine")


def moe_layer_decode(cfg, x, w_router_t, bias, w13, w13_scale, w2, w2_scale, shared_w13, shared_w13_scale,
                     shared_w2, shared_w2_scale, topk_ids, topk_weights, counts, offsets, sorted_pair,
                     pair_pos, y_perm, y_shared, out, ws, stream=None):
    c, pc = _cfg(cfg)
    _check(lib().moe_layer_decode(pc, _p(x), _p(w_router_t), _p(bias), _p(w13), _p(w13_scale), _p(w2),
                                  _p(w2_scale), _p(shared_w13), _p(shared_w13_scale), _p(shared_w2),
                                  _p(shared_w2_scale), _p(topk_ids), _p(topk_weights), _p(counts),
                                  _p(offsets), _p(sorted_pair), _p(pair_pos), _p(y_perm), _p(y_shared),
                                  _p(out), _p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_layer_decode")


def moe_quantize_fp8(rows, cols, inp, codes, scales, stream=None):
    _check(lib().moe_quantize_fp8(rows, cols, _p(inp), _p(codes), _p(scales), _stream(stream)),
           "moe_quantize_fp8")


def moe_quantize_mx(rows, cols, inp, codes, scales, stream=None):
    _check(lib().moe_quantize_mx(rows, cols, _p(inp), _p(codes), _p(scales), _stream(stream)),
           "moe_quantize_mx")


def _bad(where, why):
    raise MoEError(1, where, why)


_FLOATS = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_QUANT = {None: 0, "fp8": MOE_FP8_E4M3, "mx": MOE_MXFP4, "int8": MOE_INT8}


@functools.lru_cache(maxsize=256)
def _norm_config(*fields):
    return MoeNormConfig(*fields)


def _row_tensor(where, name, t, rows, cols, dev):
    """dtype code and row stride of a [rows, cols] fp32 or bf16 tensor on `dev` (rows may be strided)."""
    dt = _FLOATS.get(t.dtype)
    if dt is None:
        _bad(where, f"{name} must be fp32 or bf16")
    if t.shape != (rows, cols) or t.device != dev:
        _bad(where, f"{name} must be [{rows}, {cols}] on {dev}")
    st, sc = t.stride()
    if sc != 1 and cols != 1 or (st < cols and rows > 1):
        _bad(where, f"{name}: rows must not overlap and their elements must be adjacent")
    return dt, st if rows > 1 else 0


def _flat(where, name, t, dtype, n, dev):
    if t.dtype != dtype or t.numel() != n or t.device != dev or not t.is_contiguous():
        _bad(where, f"{name} must be {n} contiguous elements of {dtype} on {dev}")
    return t.data_ptr()


def _here(where, t):
    """The device of a call's tensors: the current one (a launch goes to the current device)."""
    dev = t.device
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        _bad(where, f"tensors must be on the current GPU, got {dev}")
    return dev


def moe_quantize_int8(rows, cols, inp, codes, scales, stream=None):
    """int8 rows (include/moe.h, moe_quantize_int8): inp [rows, cols] bf16, codes [rows, cols] int8, scales [rows] fp32."""
    where = "moe_quantize_int8"
    dev = _here(where, inp)
    ip = _flat(where, "inp", inp, torch.bfloat16, rows * cols, dev)
    cp = _flat(where, "codes", codes, torch.int8, rows * cols, dev)
    sp = _flat(where, "scales", scales, torch.float32, rows, dev)
    if rows:
        _check(lib().moe_quantize_int8(rows, cols, ip, cp, sp, _stream(stream)), where)


def moe_rmsnorm(x, weight, eps, y=None, residual=None, residual_out=None, quant=None, codes=None, scales=None,
                stream=None):
    """Residual addition, RMS norm and an optional 8-bit output (include/moe.h, moe_rmsnorm) on [rows, cols]
    tensors whose rows may be strided. quant: None, "fp8", "mx" or "int8", with codes [rows, cols] (uint8, int8
    for "int8") and scales ([rows, cols/128] fp32, [cols/128, rows, 4] uint8, [rows] fp32)."""
    where = "moe_rmsnorm"
    if x.dim() != 2:
        _bad(where, "x must be [rows, cols]")
    if quant not in _QUANT:
        _bad(where, f"unknown quant {quant!r}")
    dev = _here(where, x)
    rows, cols = x.shape
    xd, xs = _row_tensor(where, "x", x, rows, cols, dev)
    wd = _FLOATS.get(weight.dtype)
    if wd is None:
        _bad(where, "weight must be fp32 or bf16")
    wp = _flat(where, "weight", weight, weight.dtype, cols, dev)
    rd = yd = MOE_BF16
    rs = os_ = ys = 0
    rp = op = yp = cp = sp = None
    if residual is not None:
        rd, rs = _row_tensor(where, "residual", residual, rows, cols, dev)
        rp = residual.data_ptr()
    if residual_out is not None:
        od, os_ = _row_tensor(where, "residual_out", residual_out, rows, cols, dev)
        if residual is None or od != rd:
            _bad(where, "residual_out needs a residual of its type")
        op = residual_out.data_ptr()
    if y is not None:
        yd, ys = _row_tensor(where, "y", y, rows, cols, dev)
        yp = y.data_ptr()
    if quant is not None:
        if codes is None or scales is None:
            _bad(where, "quant needs codes and scales")
        cp = _flat(where, "codes", codes, torch.int8 if quant == "int8" else torch.uint8, rows * cols, dev)
        if quant == "mx":
            sp = _flat(where, "scales", scales, torch.uint8, rows * cols // 32, dev)
        else:
            sp = _flat(where, "scales", scales, torch.float32, rows if quant == "int8" else rows * cols // 128, dev)
    elif codes is not None or scales is not None:
        _bad(where, "codes and scales need quant")
    if rows == 0:
        return
    c = _norm_config(rows, cols, xd, rd, wd, yd, _QUANT[quant], float(eps), xs, rs, os_, ys)
    _check(lib().moe_rmsnorm(ctypes.byref(c), x.data_ptr(), wp, rp, op, yp, cp, sp, _stream(stream)), where)


def moe_gemm_int8_workspace_size() -> int:
    return int(lib().moe_gemm_int8_workspace_size())


def moe_gemm_int8(x, x_scale, w, w_scale, y, ws, offsets=None, stream=None):
    """Grouped int8 product (include/moe.h, moe_gemm_int8): x [rows, K] and w [E, N, K] (or [N, K]) int8, x_scale
    [rows] and w_scale [E, N] (or [N]) fp32, y [rows, N] fp32 or bf16 out, offsets [E + 1] int32 (E = 1: optional)."""
    where = "moe_gemm_int8"
    if x.dim() != 2 or w.dim() not in (2, 3):
        _bad(where, "x must be [rows, K], w [E, N, K] or [N, K]")
    dev = _here(where, x)
    rows, K = x.shape
    E, N = (w.shape[0] if w.dim() == 3 else 1), w.shape[-2]
    if w.shape[-1] != K:
        _bad(where, f"w rows hold {w.shape[-1]} channels, x rows {K}")
    yd = _FLOATS.get(y.dtype)
    if yd is None or y.shape != (rows, N):
        _bad(where, f"y must be [{rows}, {N}], fp32 or bf16")
    op = None if offsets is None else _flat(where, "offsets", offsets, torch.int32, E + 1, dev)
    if ws.device != dev or not ws.is_contiguous():
        _bad(where, f"ws must be a contiguous tensor on {dev}")
    xp = _flat(where, "x", x, torch.int8, rows * K, dev)
    sp = _flat(where, "x_scale", x_scale, torch.float32, rows, dev)
    wp = _flat(where, "w", w, torch.int8, E * N * K, dev)
    cp = _flat(where, "w_scale", w_scale, torch.float32, E * N, dev)
    yp = _flat(where, "y", y, y.dtype, rows * N, dev)
    if rows == 0:
        return
    _check(lib().moe_gemm_int8(E, rows, N, K, op, xp, sp, wp, cp, yp, yd, ws.data_ptr(),
                               ws.numel() * ws.element_size(), _stream(stream)), where)


def moe_get_device_error(ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    st = lib().moe_get_device_error(_p(ws), ctypes.byref(code), _stream(stream))
    if st not in (0, 5):
        _check(st, "moe_get_device_error")
    return int(code.value)


def profile_enable(on=True):
    lib().moe_profile_enable(1 if on else 0)


def profile_reset():
    lib().moe_profile_reset()


def profile_read():
    """{kernel name: (total ms, launches)} since the last reset."""
    n = lib().moe_profile_read(None, None, None, 0)
    names = (ctypes.c_char_p * max(n, 1))()
    ms = (ctypes.c_double * max(n, 1))()
    cnt = (ctypes.c_int32 * max(n, 1))()
    n = lib().moe_profile_read(names, ms, cnt, n)
    return {names[i].decode(): (ms[i], cnt[i]) for i in range(n)}
