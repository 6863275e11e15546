"""ctypes binding of libcfwd.so (include/cfwd.h), same names as the C ABI.

Argument marshalling only: every step of the convolution runs in the HIP
library.  torch is used for device memory and streams (``data_ptr()`` and
``torch.cuda.current_stream().cuda_stream``).  If the library has not been
built, loading fails loudly -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import List, NamedTuple, Optional, Sequence, Tuple, Union

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcfwd.so")

# enums (mirror include/cfwd.h)
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_NO_CANDIDATE, ERR_HIP, ERR_CACHE_IO = range(7)
LAYOUT_NCHW, LAYOUT_NCHWX, LAYOUT_NHWC = 0, 1, 2
_LAYOUTS = {"NCHW": LAYOUT_NCHW, "NCHWX": LAYOUT_NCHWX, "NHWC": LAYOUT_NHWC}
F32, BF16, I8, MXFP4 = 0, 1, 2, 3
ALGO_AUTO, ALGO_IMPLICIT_GEMM, ALGO_WINOGRAD_F2X2_3X3, ALGO_WINOGRAD_F6X6_3X3, ALGO_DIRECT, ALGO_POINTWISE = range(6)

ALGO_NAMES = {
    "auto": ALGO_AUTO, "implicit_gemm": ALGO_IMPLICIT_GEMM, "winograd_f2x2_3x3": ALGO_WINOGRAD_F2X2_3X3,
    "winograd_f6x6_3x3": ALGO_WINOGRAD_F6X6_3X3, "direct": ALGO_DIRECT, "pointwise": ALGO_POINTWISE,
}

EXPORTED = [
    "cfwd_version", "cfwd_output_dims", "cfwd_resolve_algo", "cfwd_list_candidates", "cfwd_filter_size",
    "cfwd_prepare_filter", "cfwd_workspace_size", "cfwd_scratch_size", "cfwd_conv2d_fwd", "cfwd_fastrun_select",
    "cfwd_fastrun_workspace_size", "cfwd_fastrun_lookup", "cfwd_fastrun_load", "cfwd_fastrun_save",
    "cfwd_fastrun_clear", "cfwd_fastrun_choose", "cfwd_status_string", "cfwd_last_error", "cfwd_algo_name",
    "cfwd_conv2d_fwd_noalloc", "cfwd_conv2d_fwd_ex", "cfwd_fastrun_allow_inexact_int8",
    "cfwd_bottleneck_check", "cfwd_bottleneck_filter_size", "cfwd_bottleneck_prepare", "cfwd_bottleneck_fwd",
    "cfwd_convert_layout", "cfwd_unpack_int4",
    "cfwd_mx_size", "cfwd_mx_quantize", "cfwd_mx_dequantize", "cfwd_mx_matmul_workspace_size", "cfwd_mx_matmul",
    "cfwd_gated_norm",
    "cfwd_rope_turns", "cfwd_rope", "cfwd_mx_cache_write", "cfwd_mx_cache_read",
    "cfwd_mx_cache_attention_workspace_size", "cfwd_mx_cache_attention", "cfwd_attention_workspace_size",
    "cfwd_attention",
]
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 64 << 20  # CFWD_NOALLOC_SCRATCH_BYTES


class ConvDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n", "c", "h", "w", "k", "r", "s", "stride_h", "stride_w", "pad_h",
                                            "pad_w", "dil_h", "dil_w", "groups")] + \
               [("layout", ctypes.c_int), ("x", ctypes.c_int), ("dtype", ctypes.c_int)]


class Epilogue(ctypes.Structure):
    """cfwd_epilogue: bias [K] (fp32, or int32 for int8), residual (y's shape / layout / dtype), activation."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("act", ctypes.c_int)]


class BottleneckDesc(ctypes.Structure):
    """cfwd_bottleneck_desc: x [N, C, H, W], inner channels ``mid``, output channels ``k``."""
    _fields_ = [(n, ctypes.c_int) for n in ("n", "c", "h", "w", "mid", "k")] + [("dtype", ctypes.c_int)]


class BottleneckEpilogue(ctypes.Structure):
    """cfwd_bottleneck_epilogue: fp32 biases b1 [mid], b2 [mid], b3 [K], bf16 residual, ReLU after each stage."""
    _fields_ = [("b1", ctypes.c_void_p), ("b2", ctypes.c_void_p), ("b3", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("relu1", ctypes.c_int), ("relu2", ctypes.c_int),
                ("relu3", ctypes.c_int)]


class MxMatmulDesc(ctypes.Structure):
    """cfwd_mx_matmul_desc: y [m, n] = act(x [m, k] w [n, k]^T + bias)."""
    _fields_ = [("m", ctypes.c_longlong), ("n", ctypes.c_int), ("k", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("x_stride", ctypes.c_longlong), ("act", ctypes.c_int)]


class GatedNormDesc(ctypes.Structure):
    """cfwd_gated_norm_desc: s = residual_scale * r + gate * post(b), h = pre(s) over rows of c values."""
    _fields_ = [("rows", ctypes.c_longlong), ("c", ctypes.c_int), ("rows_per_gate", ctypes.c_longlong),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("post", ctypes.c_int),
                ("pre", ctypes.c_int), ("dtype", ctypes.c_int), ("stream_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int)]


class RopeDesc(ctypes.Structure):
    """cfwd_rope_desc: rotary positions of q and k [tokens, heads, dim]."""
    _fields_ = [("tokens", ctypes.c_longlong)] + \
               [(n, ctypes.c_int) for n in ("q_heads", "k_heads", "head_dim", "pairs", "axes", "adjacent",
                                            "wide_positions", "dtype")] + \
               [(n, ctypes.c_longlong) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride",
                                                 "q_out_stride", "q_out_head_stride", "k_out_stride",
                                                 "k_out_head_stride")]


class MxCacheParts(ctypes.Structure):
    """cfwd_mx_cache: the paged cache's sizes and the addresses of its four parts."""
    _fields_ = [(n, ctypes.c_int) for n in ("pages", "page_size", "kv_heads", "head_dim")] + \
               [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")]


class MxCacheWriteDesc(ctypes.Structure):
    """cfwd_mx_cache_write_desc."""
    _fields_ = [("tokens", ctypes.c_longlong), ("dtype", ctypes.c_int), ("wide_slots", ctypes.c_int)] + \
               [(n, ctypes.c_longlong) for n in ("k_stride", "k_head_stride", "v_stride", "v_head_stride")]


class MxCacheReadDesc(ctypes.Structure):
    """cfwd_mx_cache_read_desc."""
    _fields_ = [("tokens", ctypes.c_longlong), ("sequences", ctypes.c_int), ("table_pitch", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class MxCacheAttentionDesc(ctypes.Structure):
    """cfwd_mx_cache_attention_desc."""
    _fields_ = [(n, ctypes.c_int) for n in ("sequences", "tokens", "q_heads", "table_pitch")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int)] + \
               [(n, ctypes.c_longlong) for n in ("q_seq_stride", "q_stride", "q_head_stride")]


class AttentionDesc(ctypes.Structure):
    """cfwd_attention_desc: packed prompts."""
    _fields_ = [("q_tokens", ctypes.c_longlong), ("k_tokens", ctypes.c_longlong)] + \
               [(n, ctypes.c_int) for n in ("sequences", "q_heads", "kv_heads", "head_dim", "causal")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int)] + \
               [(n, ctypes.c_longlong) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride",
                                                 "v_head_stride")]


class Algo(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("config_id", ctypes.c_int), ("median_ms", ctypes.c_float)]

    def __repr__(self):
        return "Algo(%s, ms=%.4g)" % (algo_name(self), self.median_ms)

    def key(self) -> Tuple[int, int]:
        return (self.kind, self.config_id)


class CfwdError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (_lib().cfwd_status_string(status).decode(), msg))
        self.status = status


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libcfwd.so is not built (run python -m cnn_convolution_fwd_amd.build)")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        dp = P(ConvDesc)
        lib.cfwd_version.restype = ctypes.c_char_p
        lib.cfwd_status_string.restype = ctypes.c_char_p
        lib.cfwd_status_string.argtypes = [ctypes.c_int]
        lib.cfwd_last_error.restype = ctypes.c_char_p
        lib.cfwd_algo_name.restype = ctypes.c_char_p
        lib.cfwd_algo_name.argtypes = [Algo]
        lib.cfwd_rope_turns.restype = ctypes.c_uint64
        lib.cfwd_rope_turns.argtypes = [ctypes.c_double]
        sigs = {
            "cfwd_output_dims": [dp, P(ctypes.c_int), P(ctypes.c_int)],
            "cfwd_resolve_algo": [dp, Algo, P(Algo)],
            "cfwd_list_candidates": [dp, P(Algo), ctypes.c_int, P(ctypes.c_int)],
            "cfwd_filter_size": [dp, Algo, P(sz)],
            "cfwd_prepare_filter": [dp, Algo, vp, vp, sz, vp],
            "cfwd_workspace_size": [dp, Algo, P(sz)],
            "cfwd_scratch_size": [dp, Algo, P(sz)],
            "cfwd_conv2d_fwd": [dp, Algo, vp, vp, vp, vp, vp, vp, sz, vp],
            "cfwd_conv2d_fwd_noalloc": [dp, Algo, vp, vp, vp, vp, vp, vp],
            "cfwd_conv2d_fwd_ex": [dp, Algo, vp, vp, vp, vp, P(Epilogue), vp, vp, sz, vp],
            "cfwd_fastrun_select": [dp, vp, vp, vp, vp, vp, sz, vp, P(Algo)],
            "cfwd_fastrun_workspace_size": [dp, P(sz)],
            "cfwd_fastrun_lookup": [dp, P(Algo)],
            "cfwd_fastrun_load": [ctypes.c_char_p],
            "cfwd_fastrun_save": [ctypes.c_char_p],
            "cfwd_fastrun_clear": [],
            "cfwd_fastrun_allow_inexact_int8": [ctypes.c_int],
            "cfwd_bottleneck_check": [P(BottleneckDesc)],
            "cfwd_unpack_int4": [vp, vp, ctypes.c_longlong, vp],
            "cfwd_convert_layout": [ctypes.c_int] * 4 + [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, ctypes.c_int,
                                                         ctypes.c_int, vp, vp],
            "cfwd_bottleneck_filter_size": [P(BottleneckDesc), P(sz)],
            "cfwd_bottleneck_prepare": [P(BottleneckDesc), vp, vp, sz, vp],
            "cfwd_bottleneck_fwd": [P(BottleneckDesc), vp, vp, vp, vp, P(BottleneckEpilogue), vp, vp],
            "cfwd_mx_size": [ctypes.c_longlong, ctypes.c_int, P(sz), P(sz)],
            "cfwd_mx_quantize": [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, vp, ctypes.c_longlong, vp, vp, vp],
            "cfwd_mx_dequantize": [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp],
            "cfwd_mx_matmul_workspace_size": [P(MxMatmulDesc), P(sz)],
            "cfwd_mx_matmul": [P(MxMatmulDesc)] + [vp] * 8 + [sz, vp],
            "cfwd_gated_norm": [P(GatedNormDesc)] + [vp] * 11,
            "cfwd_rope": [P(RopeDesc)] + [vp] * 7,
            "cfwd_mx_cache_write": [P(MxCacheWriteDesc), P(MxCacheParts)] + [vp] * 4,
            "cfwd_mx_cache_read": [P(MxCacheReadDesc), P(MxCacheParts)] + [vp] * 5,
            "cfwd_mx_cache_attention_workspace_size": [P(MxCacheAttentionDesc), P(MxCacheParts), P(sz)],
            "cfwd_mx_cache_attention": [P(MxCacheAttentionDesc), P(MxCacheParts)] + [vp] * 5 + [sz, vp],
            "cfwd_attention_workspace_size": [P(AttentionDesc), P(sz)],
            "cfwd_attention": [P(AttentionDesc)] + [vp] * 7 + [sz, vp],
            "cfwd_fastrun_choose": [P(Algo), P(ctypes.c_float), ctypes.c_int, ctypes.c_int, P(ctypes.c_int),
                                    P(ctypes.c_int)],
        }
        for name, args in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _LIB = lib
    return _LIB


def library():
    """The loaded ctypes library (loads it on first use)."""
    return _lib()


def _check(status: int):
    if status != OK:
        raise CfwdError(status, _lib().cfwd_last_error().decode())


# ------------------------------------------------------------ descriptors

def _pair(v) -> Tuple[int, int]:
    if isinstance(v, (tuple, list)):
        return int(v[0]), int(v[1])
    return int(v), int(v)


def make_desc(n, c, h, w, k, r, s, stride=1, padding=0, dilation=1, groups=1, layout="NCHW", x_block=None,
              dtype="f32") -> ConvDesc:
    sh, sw = _pair(stride)
    ph, pw = _pair(padding)
    dh, dw = _pair(dilation)
    lay = _LAYOUTS[layout.upper()]
    dt = {"f32": F32, "fp32": F32, "float32": F32, "bf16": BF16, "bfloat16": BF16, "i8": I8, "int8": I8}[dtype]
    return ConvDesc(n, c, h, w, k, r, s, sh, sw, ph, pw, dh, dw, groups, lay, int(x_block or 0), dt)


def algo(kind: Union[str, int] = "auto", config_id: int = -1) -> Algo:
    if isinstance(kind, str):
        kind = ALGO_NAMES[kind]
    return Algo(kind, config_id, 0.0)


def algo_name(a: Algo) -> str:
    return _lib().cfwd_algo_name(a).decode()


def version() -> str:
    return _lib().cfwd_version().decode()


def output_dims(desc: ConvDesc) -> Tuple[int, int]:
    oh, ow = ctypes.c_int(), ctypes.c_int()
    _check(_lib().cfwd_output_dims(ctypes.byref(desc), ctypes.byref(oh), ctypes.byref(ow)))
    return oh.value, ow.value


def resolve_algo(desc: ConvDesc, a: Algo) -> Algo:
    out = Algo()
    _check(_lib().cfwd_resolve_algo(ctypes.byref(desc), a, ctypes.byref(out)))
    return out


def list_candidates(desc: ConvDesc) -> List[Algo]:
    n = ctypes.c_int()
    _check(_lib().cfwd_list_candidates(ctypes.byref(desc), None, 0, ctypes.byref(n)))
    arr = (Algo * max(1, n.value))()
    _check(_lib().cfwd_list_candidates(ctypes.byref(desc), arr, n.value, ctypes.byref(n)))
    return [arr[i] for i in range(n.value)]


def filter_size(desc: ConvDesc, a: Algo) -> int:
    b = ctypes.c_size_t()
    _check(_lib().cfwd_filter_size(ctypes.byref(desc), a, ctypes.byref(b)))
    return b.value


def workspace_size(desc: ConvDesc, a: Algo) -> int:
    b = ctypes.c_size_t()
    _check(_lib().cfwd_workspace_size(ctypes.byref(desc), a, ctypes.byref(b)))
    return b.value


def scratch_size(desc: ConvDesc, a: Algo) -> int:
    b = ctypes.c_size_t()
    _check(_lib().cfwd_scratch_size(ctypes.byref(desc), a, ctypes.byref(b)))
    return b.value


def fastrun_workspace_size(desc: ConvDesc) -> int:
    b = ctypes.c_size_t()
    _check(_lib().cfwd_fastrun_workspace_size(ctypes.byref(desc), ctypes.byref(b)))
    return b.value


def fastrun_lookup(desc: ConvDesc) -> Optional[Algo]:
    out = Algo()
    st = _lib().cfwd_fastrun_lookup(ctypes.byref(desc), ctypes.byref(out))
    return out if st == OK else None


def fastrun_load(path: str):
    _check(_lib().cfwd_fastrun_load(path.encode()))


def fastrun_save(path: str):
    _check(_lib().cfwd_fastrun_save(path.encode()))


def fastrun_clear():
    _check(_lib().cfwd_fastrun_clear())


def fastrun_allow_inexact_int8(allow: bool):
    """Let int8 candidates that may differ by 1 from the exact result (int8 Winograd F(2x2)) join Fast-Run."""
    _check(_lib().cfwd_fastrun_allow_inexact_int8(1 if allow else 0))


def fastrun_choose(cands: Sequence[Algo], times: Sequence[Sequence[float]], gate_ok: Sequence[bool]) -> int:
    n = len(cands)
    reps = len(times[0]) if n else 1
    ca = (Algo * max(1, n))(*cands)
    ta = (ctypes.c_float * max(1, n * reps))(*[float(v) for row in times for v in row])
    ok = (ctypes.c_int * max(1, n))(*[int(bool(v)) for v in gate_ok])
    chosen = ctypes.c_int()
    _check(_lib().cfwd_fastrun_choose(ca, ta, n, reps, ok, ctypes.byref(chosen)))
    return chosen.value


# ---------------------------------------------------------- raw-pointer calls

def conv2d_fwd_raw(desc: ConvDesc, a: Algo, x: int, w: int, w_prepared: int, scale: int, y: int, ws: int,
                   ws_bytes: int, stream: int) -> int:
    """cfwd_conv2d_fwd with integer device pointers; returns the status."""
    return _lib().cfwd_conv2d_fwd(ctypes.byref(desc), a, x or None, w or None, w_prepared or None, scale or None,
                                  y or None, ws or None, ws_bytes, stream or None)


def epilogue_of(bias: int = 0, residual: int = 0, relu: bool = False) -> Optional[Epilogue]:
    """cfwd_epilogue from device pointers, or None when there is nothing to fuse."""
    if not bias and not residual and not relu:
        return None
    return Epilogue(bias or None, residual or None, ACT_RELU if relu else ACT_NONE)


def conv2d_fwd_ex_raw(desc: ConvDesc, a: Algo, x: int, w: int, w_prepared: int, scale: int, ep: Optional[Epilogue],
                      y: int, ws: int, ws_bytes: int, stream: int) -> int:
    """cfwd_conv2d_fwd_ex with integer device pointers; returns the status."""
    return _lib().cfwd_conv2d_fwd_ex(ctypes.byref(desc), a, x or None, w or None, w_prepared or None, scale or None,
                                     ctypes.byref(ep) if ep is not None else None, y or None, ws or None, ws_bytes,
                                     stream or None)


def conv2d_fwd_noalloc_raw(desc: ConvDesc, a: Algo, x: int, w: int, w_prepared: int, scale: int, y: int,
                           stream: int) -> int:
    """cfwd_conv2d_fwd_noalloc with integer device pointers; returns the status."""
    return _lib().cfwd_conv2d_fwd_noalloc(ctypes.byref(desc), a, x or None, w or None, w_prepared or None,
                                          scale or None, y or None, stream or None)


def prepare_filter_raw(desc: ConvDesc, a: Algo, w: int, wp: int, nbytes: int, stream: int) -> int:
    return _lib().cfwd_prepare_filter(ctypes.byref(desc), a, w or None, wp or None, nbytes, stream or None)


# ---------------------------------------------------------- torch front end

def _torch():
    import torch
    return torch


_DT = {"torch.float32": "f32", "torch.bfloat16": "bf16", "torch.int8": "i8"}


def _dtype_of(t) -> str:
    key = str(t.dtype)
    if key not in _DT:
        raise TypeError("unsupported dtype %s (float32, bfloat16 or int8)" % t.dtype)
    return _DT[key]


def desc_for(x, w, stride=1, padding=0, dilation=1, groups=1, layout="NCHW", channels=None) -> ConvDesc:
    """Descriptor for activations ``x`` (NCHW [N,C,H,W], NHWC [N,H,W,C] or NCHWX [N,CB,H,W,X]) and KCRS ``w``."""
    if layout.upper() == "NCHW":
        if x.dim() != 4:
            raise ValueError("NCHW activations must be 4-D")
        n, c, h, wd = x.shape
        xb = 0
    elif layout.upper() == "NHWC":
        if x.dim() != 4:
            raise ValueError("NHWC activations must be 4-D")
        n, h, wd, c = x.shape
        xb = 0
    else:
        if x.dim() != 5:
            raise ValueError("NCHWX activations must be 5-D [N, C/x, H, W, x]")
        n, cb, h, wd, xb = x.shape
        c = channels if channels is not None else cb * xb
        if not (cb - 1) * xb < c <= cb * xb:
            raise ValueError("channels=%d does not match %d blocks of %d" % (c, cb, xb))
    k, cg, r, s = w.shape
    if cg * groups != c:
        raise ValueError("weights [K, C/G, R, S] = %s do not match C=%d, groups=%d" % (tuple(w.shape), c, groups))
    return make_desc(n, c, h, wd, k, r, s, stride, padding, dilation, groups, layout, xb, _dtype_of(x))


def _out_shape(desc: ConvDesc):
    oh, ow = output_dims(desc)
    if desc.layout == LAYOUT_NCHW:
        return (desc.n, desc.k, oh, ow)
    if desc.layout == LAYOUT_NHWC:
        return (desc.n, oh, ow, desc.k)
    return (desc.n, -(-desc.k // desc.x), oh, ow, desc.x)


def _stream():
    torch = _torch()
    return torch.cuda.current_stream().cuda_stream


def _check_dev(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def prepare_filter(w, desc: ConvDesc, a: Algo):
    """Prepared filter of algorithm ``a`` as a uint8 device tensor (None if it reads KCRS)."""
    torch = _torch()
    a = resolve_algo(desc, a)
    nbytes = filter_size(desc, a)
    if nbytes == 0:
        return None
    _check_dev(w)
    wp = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _check(prepare_filter_raw(desc, a, w.data_ptr(), wp.data_ptr(), nbytes, _stream()))
    return wp


def conv2d_fwd(x, w, stride=1, padding=0, dilation=1, groups=1, layout="NCHW", channels=None, algo_kind="auto",
               config_id=-1, requant_scale=None, out=None, w_prepared=None, workspace=None, bias=None, residual=None,
               relu=False):
    """y = conv(x, w) on the current stream.  Tensors on the GPU, contiguous.

    ``algo_kind`` is one of auto, implicit_gemm, winograd_f2x2_3x3,
    winograd_f6x6_3x3, direct, pointwise; ``requant_scale`` (float32 [K]) is
    required for int8.  ``w_prepared`` is the output of ``prepare_filter`` for
    the same resolved algorithm.  ``bias`` (float32 [K], int32 for int8),
    ``residual`` (shaped like the output) and ``relu`` are the fused epilogue.
    """
    torch = _torch()
    _check_dev(x, w, requant_scale, out, w_prepared, workspace, bias, residual)
    desc = desc_for(x, w, stride, padding, dilation, groups, layout, channels)
    a = resolve_algo(desc, algo(algo_kind, config_id))
    if out is None:
        out = torch.empty(_out_shape(desc), dtype=x.dtype, device=x.device)
    ws_bytes = workspace_size(desc, a) if w_prepared is None else scratch_size(desc, a)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
    ep = epilogue_of(bias.data_ptr() if bias is not None else 0,
                     residual.data_ptr() if residual is not None else 0, relu)
    st = conv2d_fwd_ex_raw(desc, a, x.data_ptr(), w.data_ptr(),
                           w_prepared.data_ptr() if w_prepared is not None else 0,
                           requant_scale.data_ptr() if requant_scale is not None else 0, ep, out.data_ptr(),
                           workspace.data_ptr() if workspace is not None else 0, ws_bytes, _stream())
    _check(st)
    return out


def fastrun_select(x, w, stride=1, padding=0, dilation=1, groups=1, layout="NCHW", channels=None,
                   requant_scale=None, out=None, workspace=None) -> Tuple[Algo, object]:
    """Run the Fast-Run selection for this problem; returns (best algo, output).

    ``workspace`` (uint8 device tensor of at least ``fastrun_workspace_size``
    bytes) is allocated here when not given.
    """
    torch = _torch()
    _check_dev(x, w, requant_scale, out, workspace)
    desc = desc_for(x, w, stride, padding, dilation, groups, layout, channels)
    if out is None:
        out = torch.empty(_out_shape(desc), dtype=x.dtype, device=x.device)
    nbytes = fastrun_workspace_size(desc)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    best = Algo()
    _check(_lib().cfwd_fastrun_select(ctypes.byref(desc), x.data_ptr(), w.data_ptr(),
                                      requant_scale.data_ptr() if requant_scale is not None else None,
                                      out.data_ptr(), workspace.data_ptr(), nbytes, _stream(),
                                      ctypes.byref(best)))
    return best, out


class LayerPlan:
    """One conv layer set up the way an inference step runs it.

    ``algo="auto"``: unless the map already holds the problem, the Fast-Run
    selection phase runs once on (x, w) and records its choice in the map;
    launches then pass AUTO, so the library dispatches from the map
    (execution phase).  Otherwise the named family
    (and config, "family/cfg") is resolved once and passed explicitly.  The
    filter is prepared once (constant weights) and the algorithm's scratch is
    allocated once; ``prepare_ms`` is the prepare step's device time.
    """

    def __init__(self, x, w, stride=1, padding=0, dilation=1, groups=1, layout="NCHW", channels=None,
                 requant_scale=None, algo_spec="auto", bias=None, relu=False):
        torch = _torch()
        _check_dev(x, w, requant_scale, bias)
        self.w, self.scale = w, requant_scale
        self.bias, self.relu = bias, relu  # fused epilogue (a residual is given per launch)
        self.desc = desc_for(x, w, stride, padding, dilation, groups, layout, channels)
        self.out_shape = _out_shape(self.desc)
        self.dtype, self.device = x.dtype, x.device
        if algo_spec == "auto":
            # a problem already in the map (an earlier layer of the same shape,
            # or a map loaded from a file) is dispatched from it unsearched
            best = fastrun_lookup(self.desc)
            if best is None:
                best, _ = fastrun_select(x, w, stride, padding, dilation, groups, layout, channels,
                                         requant_scale=requant_scale)
            self.chosen = resolve_algo(self.desc, algo())
            if self.chosen.key() != best.key():
                raise RuntimeError("AUTO resolves to %s, Fast-Run chose %s" % (algo_name(self.chosen),
                                                                               algo_name(best)))
            self.chosen.median_ms = best.median_ms
            self.algo_arg = algo()
        else:
            fam, _, cid = algo_spec.partition("/")
            self.chosen = resolve_algo(self.desc, algo(fam, int(cid) if cid else -1))
            self.algo_arg = self.chosen
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        self.wp = prepare_filter(w, self.desc, self.chosen)
        e1.record()
        torch.cuda.synchronize()
        self.prepare_ms = e0.elapsed_time(e1) if self.wp is not None else 0.0
        self.scratch_bytes = scratch_size(self.desc, self.chosen)
        self.scratch = torch.empty(max(self.scratch_bytes, 16), dtype=torch.uint8, device=x.device)

    @property
    def name(self) -> str:
        return algo_name(self.chosen)

    def new_output(self):
        return _torch().empty(self.out_shape, dtype=self.dtype, device=self.device)

    def launch_raw(self, x_ptr: int, y_ptr: int, stream: int, residual_ptr: int = 0) -> int:
        """Enqueue the layer on ``stream`` with raw device pointers; returns the status."""
        ep = epilogue_of(self.bias.data_ptr() if self.bias is not None else 0, residual_ptr, self.relu)
        return conv2d_fwd_ex_raw(self.desc, self.algo_arg, x_ptr, self.w.data_ptr(),
                                 self.wp.data_ptr() if self.wp is not None else 0,
                                 self.scale.data_ptr() if self.scale is not None else 0, ep, y_ptr,
                                 self.scratch.data_ptr() if self.scratch_bytes else 0, self.scratch_bytes, stream)

    def __call__(self, x, out=None, residual=None):
        """y = conv(x) (+ the fused epilogue) on the current stream (x shaped and typed like the set-up input)."""
        _check_dev(x, out, residual)
        if out is None:
            out = self.new_output()
        _check(self.launch_raw(x.data_ptr(), out.data_ptr(), _stream(),
                               residual.data_ptr() if residual is not None else 0))
        return out


# ------------------------------------------------------- fused bottleneck block

_DTYPE_CODES = {"f32": F32, "fp32": F32, "float32": F32, "bf16": BF16, "bfloat16": BF16, "i8": I8, "int8": I8}


def bottleneck_desc(n, c, h, w, mid, k, dtype="bf16") -> BottleneckDesc:
    return BottleneckDesc(n, c, h, w, mid, k, _DTYPE_CODES[dtype] if isinstance(dtype, str) else dtype)


def bottleneck_check(desc: BottleneckDesc) -> None:
    """Raise CfwdError (UNSUPPORTED with the reason) unless the fused kernel runs this block."""
    _check(_lib().cfwd_bottleneck_check(ctypes.byref(desc)))


def bottleneck_filter_size(desc: BottleneckDesc) -> int:
    b = ctypes.c_size_t()
    _check(_lib().cfwd_bottleneck_filter_size(ctypes.byref(desc), ctypes.byref(b)))
    return b.value


def bottleneck_desc_for(x, w1, w3) -> BottleneckDesc:
    n, c, h, wd = x.shape
    return bottleneck_desc(n, c, h, wd, w1.shape[0], w3.shape[0], _dtype_of(x))


def bottleneck_prepare(w2, desc: BottleneckDesc):
    """Prepared 3x3 weights of the block (uint8 device tensor)."""
    torch = _torch()
    _check_dev(w2)
    nbytes = bottleneck_filter_size(desc)
    wp = torch.empty(nbytes, dtype=torch.uint8, device=w2.device)
    _check(_lib().cfwd_bottleneck_prepare(ctypes.byref(desc), w2.data_ptr(), wp.data_ptr(), nbytes, _stream()))
    return wp


def bottleneck_fwd_raw(desc: BottleneckDesc, x: int, w1: int, w2p: int, w3: int, ep, y: int, stream) -> int:
    """cfwd_bottleneck_fwd with integer device pointers; returns the status."""
    return _lib().cfwd_bottleneck_fwd(ctypes.byref(desc), x, w1, w2p, w3, ctypes.byref(ep) if ep is not None else None,
                                      y, stream)


def bottleneck_fwd(x, w1, w2_prepared, w3, b1=None, b2=None, b3=None, residual=None, relu=(False, False, False),
                   out=None):
    """y = the fused bottleneck block of NCHW ``x`` on the current stream (see cfwd.h)."""
    torch = _torch()
    _check_dev(x, w1, w2_prepared, w3, b1, b2, b3, residual, out)
    desc = bottleneck_desc_for(x, w1, w3)
    if out is None:
        out = torch.empty((desc.n, desc.k, desc.h, desc.w), dtype=x.dtype, device=x.device)
    ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    ep = BottleneckEpilogue(ptr(b1), ptr(b2), ptr(b3), ptr(residual), int(bool(relu[0])), int(bool(relu[1])),
                            int(bool(relu[2])))
    _check(bottleneck_fwd_raw(desc, x.data_ptr(), w1.data_ptr(), w2_prepared.data_ptr(), w3.data_ptr(), ep,
                              out.data_ptr(), _stream()))
    return out


# ------------------------------------------------------- layout conversion

def convert_layout(t, src_layout: str, dst_layout: str, dst_x: int = 0, channels: Optional[int] = None, out=None):
    """Copy activations between NCHW [N,C,H,W], NHWC [N,H,W,C] and NCHWX [N,CB,H,W,X] (cfwd_convert_layout)."""
    torch = _torch()
    _check_dev(t, out)
    sl, dl = src_layout.upper(), dst_layout.upper()
    if sl == "NCHW":
        n, c, h, w = t.shape
        sx = 0
    elif sl == "NHWC":
        n, h, w, c = t.shape
        sx = 0
    else:
        n, cb, h, w, sx = t.shape
        c = channels if channels is not None else cb * sx
    shape = {"NCHW": (n, c, h, w), "NHWC": (n, h, w, c)}.get(dl) or (n, -(-c // dst_x), h, w, dst_x)
    if out is None:
        out = torch.empty(shape, dtype=t.dtype, device=t.device)
    _check(_lib().cfwd_convert_layout(n, c, h, w, _DTYPE_CODES[_dtype_of(t)], _LAYOUTS[sl], sx, t.data_ptr(),
                                      _LAYOUTS[dl], int(dst_x), out.data_ptr(), _stream()))
    return out


# ------------------------------------------------------- 4-bit weights

def unpack_int4(packed, count: int, out=None):
    """int8 tensor of ``count`` signed 4-bit values packed two per byte, low nibble first (cfwd_unpack_int4)."""
    torch = _torch()
    _check_dev(packed, out)
    if out is None:
        out = torch.empty(count, dtype=torch.int8, device=packed.device)
    _check(_lib().cfwd_unpack_int4(packed.data_ptr(), out.data_ptr(), int(count), _stream()))
    return out


# ------------------------------------------------------- MXFP4 and the feed-forward block

_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU}
_NORMS = {"none": NORM_NONE, "rms": NORM_RMS, "layer": NORM_LAYER}
_MX_CODES = {**{k: v for k, v in _DTYPE_CODES.items() if v != I8}, "mx": MXFP4, "mxfp4": MXFP4}


class MxTensor(NamedTuple):
    """Rows in microscaled 4-bit floating point (format: cfwd.h): ``codes`` uint8 [..., 16 * ceil(cols / 32)],
    ``scales`` uint8 [..., ceil(cols / 32) rounded up to 4], of which the bytes past the blocks do not count,
    ``cols`` values a row."""
    codes: object
    scales: object
    cols: int

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.cols)


def mx_pitches(cols: int) -> Tuple[int, int]:
    """Bytes of a row's codes and of its scales."""
    kb = -(-cols // 32)
    return 16 * kb, -(-kb // 4) * 4


def _code(table, key, what: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError("unknown %s %r (one of %s)" % (what, key, ", ".join(sorted(table)))) from None


def _float_code(t) -> int:
    code = _DTYPE_CODES[_dtype_of(t)]
    if code == I8:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)
    return code


def _rows_of(t) -> Tuple[int, int, int]:
    """(rows, values a row, row pitch) of a tensor whose last axis is dense and whose rows are evenly spaced."""
    shape = t.shape
    if not shape:
        raise ValueError("a tensor with at least one axis is needed")
    k = shape[-1]
    if t.is_contiguous():
        return (t.numel() // k if k else 0), k, k
    if len(shape) != 2:
        try:
            t = t.view(-1, k)
        except RuntimeError:
            raise ValueError("the rows of a tensor of strides %s are not evenly spaced" % (t.stride(),)) from None
    rows, stride = t.shape[0], t.stride(0)
    if (k > 1 and t.stride(1) != 1) or (rows > 1 and stride < k):
        raise ValueError("rows must be dense and must not overlap")
    return rows, k, stride if rows > 1 else k


def _check_on(dev: int, *ts):
    """Every tensor that is given is on GPU ``dev`` (-1: the first one was on none) and dense."""
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    for t in ts:
        if t is not None:
            if t.get_device() != dev:
                raise ValueError("tensors must be on one GPU")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _check_mx(t: MxTensor, what: str) -> int:
    """Rows of an MxTensor whose parts fit each other."""
    if not isinstance(t, MxTensor):
        raise TypeError("%s must be an MxTensor" % what)
    codes, scales, cols = t
    u8 = _torch().uint8
    if codes.dtype != u8 or scales.dtype != u8:
        raise TypeError("%s: codes and scales must be uint8" % what)
    cs, ss = codes.shape, scales.shape
    cp, sp = mx_pitches(cols)
    if not cp or cs[-1] != cp or ss[-1] != sp or cs[:-1] != ss[:-1]:
        raise ValueError("%s: codes %s and scales %s do not hold rows of %d values"
                         % (what, tuple(cs), tuple(ss), cols))
    return codes.numel() // cp


def _guard(dev: int):
    """None when ``dev`` is the current GPU, else a context that makes it that (kernels go to the current GPU's stream)."""
    torch = _torch()
    return None if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _stream_of(dev: int) -> int:
    """Handle of the current stream of GPU ``dev``; the plain call behind torch.cuda.current_stream, 2.7 us cheaper."""
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _new_mx(lead, cols: int, device) -> MxTensor:
    torch = _torch()
    cp, sp = mx_pitches(cols)
    return MxTensor(torch.empty((*lead, cp), dtype=torch.uint8, device=device),
                    torch.empty((*lead, sp), dtype=torch.uint8, device=device), cols)


def _check_mx_out(t: MxTensor, shape):
    _check_mx(t, "out")
    if tuple(t.shape) != tuple(shape):
        raise ValueError("out must hold %s values" % (tuple(shape),))


def mx_quantize(x, out: Optional[MxTensor] = None) -> MxTensor:
    """x [..., k] (float32 / bfloat16, rows evenly spaced) in MXFP4 (cfwd_mx_quantize)."""
    dev = x.get_device()
    rows, k, stride = _rows_of(x)
    code = _float_code(x)
    if out is None:
        _check_on(dev)
        out = _new_mx(x.shape[:-1], k, x.device)
    else:
        _check_mx_out(out, x.shape)
        _check_on(dev, out.codes, out.scales)
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return mx_quantize(x, out)
    _check(_lib().cfwd_mx_quantize(rows, k, code, x.data_ptr(), stride, out.codes.data_ptr(), out.scales.data_ptr(),
                                   _stream_of(dev)))
    return out


def mx_dequantize(t: MxTensor, dtype="f32", out=None):
    """The values of an MXFP4 tensor in float32 or bfloat16, both exact (cfwd_mx_dequantize)."""
    torch = _torch()
    rows = _check_mx(t, "the tensor")
    dev = t.codes.get_device()
    if out is None:
        code = _code(_MX_CODES, dtype, "dtype")
        if code == MXFP4:
            raise ValueError("dtype must be f32 or bf16")
        out = torch.empty(t.shape, dtype=torch.float32 if code == F32 else torch.bfloat16, device=t.codes.device)
    elif tuple(out.shape) != tuple(t.shape):
        raise ValueError("out must have the shape %s" % (tuple(t.shape),))
    else:
        code = _float_code(out)
    _check_on(dev, t.codes, t.scales, out)
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return mx_dequantize(t, out=out)
    _check(_lib().cfwd_mx_dequantize(rows, t.cols, code, t.codes.data_ptr(), t.scales.data_ptr(), out.data_ptr(),
                                     _stream_of(dev)))
    return out


@functools.lru_cache(maxsize=1024)
def _mx_matmul_desc(dev, *sizes):
    """(descriptor reference, workspace bytes) of a product of these sizes on GPU ``dev``, the current one, whose
    number of CUs decides about the workspace; made once, read only."""
    desc = MxMatmulDesc(*sizes)
    return ctypes.byref(desc), mx_matmul_workspace_size(desc)


@functools.lru_cache(maxsize=1024)
def _gated_norm_desc(*sizes):
    return ctypes.byref(GatedNormDesc(*sizes))


def mx_matmul_workspace_size(desc: MxMatmulDesc) -> int:
    b = ctypes.c_size_t()
    _check(_lib().cfwd_mx_matmul_workspace_size(ctypes.byref(desc), ctypes.byref(b)))
    return b.value


def mx_matmul(x, w: MxTensor, bias=None, act: str = "none", out_dtype=None, out=None, workspace=None):
    """act(x w^T + bias): x [..., k] against MXFP4 weights [n, k] (cfwd_mx_matmul).

    ``x`` is an MxTensor, or float32 / bfloat16 and then quantised by the call
    exactly as ``mx_quantize`` does.  A 1x1 convolution of NHWC activations is
    this product with its channels as the rows.  ``act``: none, relu, silu or
    gelu (the form with tanh); ``bias`` float32 [n].  ``out_dtype``: f32, bf16
    or mx (default: x's own, bf16 for an MxTensor).  ``workspace`` (uint8,
    ``mx_matmul_workspace_size`` bytes) is allocated when not given.
    """
    torch = _torch()
    n = _check_mx(w, "w")
    w_codes, w_scales, k = w
    if w_codes.dim() != 2:
        raise ValueError("w must be a matrix [n, k]")
    if isinstance(x, MxTensor):
        rows, stride, x_code = _check_mx(x, "x"), k, MXFP4
        xt, x_scales, x_k = x
        lead, dev = xt.shape[:-1], xt.get_device()
        _check_on(dev, xt, x_scales, w_codes, w_scales, bias, workspace)
        xs = x_scales.data_ptr()
    else:
        xt, xs = x, None
        rows, x_k, stride = _rows_of(x)
        x_code, lead, dev = _float_code(x), x.shape[:-1], x.get_device()
        _check_on(dev, w_codes, w_scales, bias, workspace)
    if x_k != k:
        raise ValueError("x has rows of %d values, w of %d" % (x_k, k))
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (n,)):
        raise ValueError("bias must be float32 [%d]" % n)
    y_code = _code(_MX_CODES, out_dtype, "out_dtype") if out_dtype is not None else None
    if out is None:
        if y_code is None:
            y_code = BF16 if x_code == MXFP4 else x_code
        out = _new_mx(lead, n, xt.device) if y_code == MXFP4 else torch.empty(
            (*lead, n), dtype=torch.float32 if y_code == F32 else torch.bfloat16, device=xt.device)
    else:
        if isinstance(out, MxTensor):
            _check_mx_out(out, (*lead, n))
            code = MXFP4
            _check_on(dev, out.codes, out.scales)
        else:
            if tuple(out.shape) != (*lead, n):
                raise ValueError("out must have the shape %s" % ((*lead, n),))
            code = _float_code(out)
            _check_on(dev, out)
        if y_code is not None and y_code != code:
            raise ValueError("out is not of out_dtype")
        y_code = code
    act_code = _code(_ACTS, act, "act")
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return mx_matmul(x, w, bias, act, None, out, workspace)
    desc, ws_bytes = _mx_matmul_desc(dev, rows, n, k, x_code, y_code, stride, act_code)
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=xt.device)
        ws = workspace.data_ptr()
    else:
        ws = None
    yp, ys = (out.codes.data_ptr(), out.scales.data_ptr()) if y_code == MXFP4 else (out.data_ptr(), None)
    _check(_lib().cfwd_mx_matmul(desc, xt.data_ptr(), xs, w_codes.data_ptr(), w_scales.data_ptr(),
                                 _ptr(bias), yp, ys, ws, ws_bytes, _stream_of(dev)))
    return out


def gated_norm(b, residual=None, gate=None, residual_scale: float = 1.0, post: str = "none", post_weight=None,
               post_bias=None, pre: str = "rms", pre_weight=None, pre_bias=None, eps: float = 1e-6, out_dtype=None,
               sum_out=None, out=None, want_sum: bool = True):
    """(s, h): s = residual_scale * residual + gate * post(b), h = pre(s) over the last axis (cfwd_gated_norm).

    ``b`` (float32 / bfloat16 [..., c], or None: its norm counts as 0, so post(b) is
    ``post_bias``) is a block's output, ``residual`` (b's dtype, or float32) the residual stream.  ``gate``
    [g, c] or [c] has one row for each run of ceil(rows / g) rows (images,
    sequences).  ``post`` and ``pre``: none, rms or layer, with float32 [c]
    weights and biases.  h is in b's dtype, or an MxTensor for ``out_dtype``
    "mx", ready for ``mx_matmul``; without b and gate it may be float32 or
    bfloat16 as ``out_dtype`` says; ``pre`` "none" gives h = None.  s is
    written to ``sum_out`` (which may be ``residual``); ``want_sum`` False: not at all.
    """
    torch = _torch()
    like = b if b is not None else residual
    if like is None:
        raise ValueError("b and residual must not both be None")
    dev, shape = like.get_device(), like.shape
    if not shape:
        raise ValueError("a tensor with at least one axis is needed")
    _check_on(dev, b, residual, gate, post_weight, post_bias, pre_weight, pre_bias, sum_out)
    c = shape[-1]
    rows = like.numel() // c if c else 0
    if b is not None and residual is not None and residual.shape != shape:
        raise ValueError("b and residual must have one shape")
    b_code = _float_code(b if b is not None else gate if gate is not None else like)
    stream_like = residual if residual is not None else sum_out
    s_code = b_code if stream_like is None else _float_code(stream_like)
    per = 0
    if gate is not None:
        if _float_code(gate) != b_code or gate.dim() not in (1, 2) or gate.shape[-1] != c:
            raise ValueError("gate must be [groups, %d] of b's dtype" % c)
        groups = gate.shape[0] if gate.dim() == 2 else 1
        if groups == 0 and rows:
            raise ValueError("gate has no rows")
        per = -(-rows // groups) if groups else 0
    for t in (post_weight, post_bias, pre_weight, pre_bias):
        if t is not None and (t.dtype != torch.float32 or t.shape != (c,)):
            raise ValueError("weights and biases must be float32 [%d]" % c)
    post_code, pre_code = _code(_NORMS, post, "norm"), _code(_NORMS, pre, "norm")
    h_code = b_code if out_dtype is None else _code(_MX_CODES, out_dtype, "out_dtype")
    if out is not None:
        if pre_code == NORM_NONE:
            raise ValueError("pre none has no h to write to out")
        code = MXFP4 if isinstance(out, MxTensor) else _float_code(out)
        if out_dtype is not None and code != h_code:
            raise ValueError("out is not of out_dtype")
        h_code = code
        if code == MXFP4:
            _check_mx_out(out, shape)
            _check_on(dev, out.codes, out.scales)
        else:
            if out.shape != shape:
                raise ValueError("out must have the shape %s" % (tuple(shape),))
            _check_on(dev, out)
    if b is None and gate is None and h_code != MXFP4:
        b_code = h_code  # nothing else has b's dtype
    if sum_out is not None:
        if sum_out.shape != shape or _float_code(sum_out) != s_code:
            raise ValueError("sum_out must have residual's shape and dtype")
    elif want_sum or pre_code == NORM_NONE:
        sum_out = torch.empty_like(stream_like if stream_like is not None else like)
    if pre_code == NORM_NONE:
        out, h_code = None, b_code
    elif out is None:
        if h_code == MXFP4:
            out = _new_mx(shape[:-1], c, like.device)
        else:
            out = torch.empty_like(like) if b is not None else torch.empty(
                shape, dtype=torch.float32 if h_code == F32 else torch.bfloat16, device=like.device)
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return gated_norm(b, residual, gate, residual_scale, post, post_weight, post_bias, pre, pre_weight,
                              pre_bias, eps, out_dtype, sum_out, out, want_sum)
    # as numbers: a tensor would be kept, and found again, as the object that it is
    desc = _gated_norm_desc(rows, c, per, float(residual_scale), float(eps), post_code, pre_code, b_code, s_code,
                            h_code)
    hp, hs = (out.codes.data_ptr(), out.scales.data_ptr()) if h_code == MXFP4 else (_ptr(out), None)
    _check(_lib().cfwd_gated_norm(desc, _ptr(b), _ptr(residual), _ptr(gate), _ptr(post_weight),
                                  _ptr(post_bias), _ptr(pre_weight), _ptr(pre_bias), _ptr(sum_out), hp, hs,
                                  _stream_of(dev)))
    return sum_out, out


# ------------------------------------------------------- rotary positions, the MXFP4 cache and attention

class RopeTable(NamedTuple):
    """Rotary positions' axes and frequencies (``rope_table``): ``pairs`` int64 [pairs, 2] on the GPU, ``axes``."""
    pairs: object
    axes: int


_ROPE_ORDERS = ("runs", "turns", "each")


def rope_table(rotary_dim: int, sections: Optional[Sequence[int]] = None, base: float = 10000.0, order: str = "runs",
               frequencies: Optional[Sequence[float]] = None, device="cuda") -> RopeTable:
    """Axis and frequency of each of ``rotary_dim / 2`` pairs, for ``rope``; made once.

    ``sections``: pairs of each axis (time, height, width, ...), rotary_dim / 2
    in all; default one axis.  ``order`` "runs": the first section's pairs belong
    to axis 0, the next ones to axis 1, ..., and the frequencies
    base^(-2 i / rotary_dim) run on over all pairs i; "turns": the axes take
    turns pair by pair until their sections are used up, with the same
    frequencies; "each": as "runs", but every axis has frequencies of its own,
    base^(-i / n) for its n pairs.  ``frequencies`` (radians a position, one for
    each pair) take the place of these powers of ``base``.
    """
    torch = _torch()
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    pairs = rotary_dim // 2
    sections = [pairs] if sections is None else [int(n) for n in sections]
    if not sections or min(sections) < 0 or sum(sections) != pairs:
        raise ValueError("sections must be %d pairs in all" % pairs)
    if order not in _ROPE_ORDERS:
        raise ValueError("unknown order %r (one of %s)" % (order, ", ".join(_ROPE_ORDERS)))
    if order == "turns":
        rounds = range(max(sections))
        axes = [a for i in rounds for a, n in enumerate(sections) if i < n]
    else:
        axes = [a for a, n in enumerate(sections) for _ in range(n)]
    if frequencies is not None:
        freq = [float(f) for f in frequencies]
        if len(freq) != pairs:
            raise ValueError("frequencies must be %d numbers" % pairs)
    elif order == "each":
        freq = [float(base) ** (-i / n) for n in sections for i in range(n)]
    else:
        freq = [float(base) ** (-i / pairs) for i in range(pairs)]
    turns = [_lib().cfwd_rope_turns(f) for f in freq]
    signed = [t - (1 << 64) if t >> 63 else t for t in turns]
    table = torch.tensor([[t, a] for t, a in zip(signed, axes)], dtype=torch.int64).reshape(pairs, 2)
    return RopeTable(table.to(device), len(sections))


def _int_code(t, what: str) -> int:
    """0 for an int32 tensor, 1 for int64."""
    torch = _torch()
    if t.dtype == torch.int32:
        return 0
    if t.dtype == torch.int64:
        return 1
    raise TypeError("%s must be int32 or int64" % what)


def _int32(dev: int, t, shape, what: str):
    if t.dtype != _torch().int32 or t.shape != shape:
        raise ValueError("%s must be int32 %s" % (what, list(shape)))
    _check_on(dev, t)


# Outputs are allocated with new_empty from a plain tuple, 0.9 us a tensor under torch.empty with dtype and device named.

def _heads_of(t, what: str) -> Tuple[int, int, int, int, int]:
    """(tokens, heads, dim, token stride, head stride) of [tokens, heads, dim] with dense dims; the stride of an axis of
    one, which may be any number, as in a dense tensor."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must be [tokens, heads, dim]" % what)
    st, sh, sd = t.stride()
    if sd != 1 and shape[2] > 1:
        raise ValueError("the last axis of %s must be dense" % what)
    tokens, heads, dim = shape
    return tokens, heads, dim, st if tokens > 1 else heads * dim, sh if heads > 1 else dim


@functools.lru_cache(maxsize=1024)
def _rope_desc(*sizes):
    return ctypes.byref(RopeDesc(*sizes))


def rope(q, k, positions, table: RopeTable, adjacent: bool = False, q_out=None, k_out=None):
    """(q, k) turned by their positions (cfwd_rope).

    ``q`` [tokens, heads, dim] and ``k`` (the same with its own number of heads,
    or None) are float32 or bfloat16 with dense dims; tokens and heads may be
    strided, as parts of one projection's output are.  ``positions``: int32 or
    int64 [tokens, axes] (or [tokens] for one axis).  ``adjacent``: pairs are values
    2 i and 2 i + 1 of a head instead of i and i + rotary_dim / 2.  ``q_out`` and
    ``k_out`` may be ``q`` and ``k`` themselves.
    """
    torch = _torch()
    dev = q.get_device()
    tokens, heads, dim, qs, qh = _heads_of(q, "q")
    code = _float_code(q)
    if q_out is None:
        q_out, qos, qoh = q.new_empty((tokens, heads, dim)), heads * dim, dim
    elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.get_device() != dev:
        raise ValueError("q_out must be as q")
    else:
        _, _, _, qos, qoh = _heads_of(q_out, "q_out")
    kh = ks = khs = kos = koh = 0
    if k is not None:
        kt, kh, kd, ks, khs = _heads_of(k, "k")
        if kt != tokens or kd != dim or k.dtype != q.dtype or k.get_device() != dev:
            raise ValueError("k must have q's tokens, dim, dtype and device")
        if k_out is None:
            k_out, kos, koh = k.new_empty((tokens, kh, dim)), kh * dim, dim
        elif k_out.shape != k.shape or k_out.dtype != k.dtype or k_out.get_device() != dev:
            raise ValueError("k_out must be as k")
        else:
            _, _, _, kos, koh = _heads_of(k_out, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    pairs, axes = table
    if positions.shape != (tokens, axes) and not (axes == 1 and positions.shape == (tokens,)):
        raise ValueError("positions must be [%d, %d]" % (tokens, axes))
    wide = _int_code(positions, "positions")
    if pairs.dtype != torch.int64 or pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("table must come from rope_table")
    _check_on(dev, positions, pairs)
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return rope(q, k, positions, table, adjacent, q_out, k_out)
    desc = _rope_desc(tokens, heads, kh, dim, pairs.shape[0], axes, int(bool(adjacent)), wide, code, qs, qh, ks, khs,
                      qos, qoh, kos, koh)
    _check(_lib().cfwd_rope(desc, q.data_ptr(), _ptr(k), positions.data_ptr(), pairs.data_ptr(), q_out.data_ptr(),
                            _ptr(k_out), _stream_of(dev)))
    return q_out, k_out


class MxCache(NamedTuple):
    """A paged cache of keys and values: ``k`` and ``v`` are MxTensors [pages, heads, page_size, dim].  Token t of a
    sequence is row t % page_size of the page that its page table names at t // page_size."""
    k: MxTensor
    v: MxTensor


def mx_cache(pages: int, page_size: int, heads: int, dim: int, device="cuda") -> MxCache:
    """An MxCache whose values are all 0."""
    torch = _torch()
    cp, sp = mx_pitches(dim)
    zeros = lambda pitch: torch.zeros(pages, heads, page_size, pitch, dtype=torch.uint8, device=device)  # noqa: E731
    return MxCache(MxTensor(zeros(cp), zeros(sp), dim), MxTensor(zeros(cp), zeros(sp), dim))


def _check_cache(cache: MxCache):
    """(GPU, sizes (pages, page_size, heads, dim), descriptor of the cache) of one whose parts fit each other."""
    if not isinstance(cache, MxCache):
        raise TypeError("cache must be an MxCache")
    (kc, ks, dim), (vc, vs, v_dim) = cache
    shape, u8 = kc.shape, _torch().uint8
    if len(shape) != 4:
        raise ValueError("the cache's parts must be MxTensors [pages, heads, page_size, dim] of one shape")
    pages, heads, page_size, pitch = shape
    cp, sp = mx_pitches(dim)
    if v_dim != dim or vc.shape != shape or pitch != cp or not cp or ks.shape != (pages, heads, page_size, sp) \
            or vs.shape != ks.shape:
        raise ValueError("the cache's parts must be MxTensors [pages, heads, page_size, dim] of one shape")
    if kc.dtype != u8 or ks.dtype != u8 or vc.dtype != u8 or vs.dtype != u8:
        raise TypeError("codes and scales must be uint8")
    dev = kc.get_device()
    _check_on(dev, kc, ks, vc, vs)
    return dev, (pages, page_size, heads, dim), ctypes.byref(MxCacheParts(
        pages, page_size, heads, dim, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr()))


@functools.lru_cache(maxsize=1024)
def _mx_cache_write_desc(*sizes):
    return ctypes.byref(MxCacheWriteDesc(*sizes))


def mx_cache_write(k, v, cache: MxCache, slots):
    """Quantises ``k`` and ``v`` [tokens, heads, dim] into the cache (cfwd_mx_cache_write).

    float32 or bfloat16 with dense dims, tokens and heads may be strided.
    ``slots`` (int32 or int64 [tokens]): page * page_size + offset of each token; one
    that is negative, or past the cache, leaves its token out.  Slots must differ from each other.
    """
    dev, sizes, parts = _check_cache(cache)
    tokens, heads, dim, ks, kh = _heads_of(k, "k")
    vt, vheads, vd, vs, vh = _heads_of(v, "v")
    if (heads, dim) != sizes[2:] or (vt, vheads, vd) != (tokens, heads, dim) or v.dtype != k.dtype:
        raise ValueError("k and v must be [tokens, %d, %d] of one dtype" % sizes[2:])
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    code, wide = _float_code(k), _int_code(slots, "slots")
    if slots.shape != (tokens,):
        raise ValueError("slots must be [%d]" % tokens)
    _check_on(dev, slots)
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return mx_cache_write(k, v, cache, slots)
    _check(_lib().cfwd_mx_cache_write(_mx_cache_write_desc(tokens, code, wide, ks, kh, vs, vh), parts, k.data_ptr(),
                                      v.data_ptr(), slots.data_ptr(), _stream_of(dev)))


@functools.lru_cache(maxsize=1024)
def _mx_cache_read_desc(*sizes):
    return ctypes.byref(MxCacheReadDesc(*sizes))


def _check_table(dev: int, table) -> Tuple[int, int]:
    if table.dtype != _torch().int32 or table.dim() != 2:
        raise ValueError("page_table must be int32 [sequences, pages]")
    _check_on(dev, table)
    return table.shape


def mx_cache_read(cache: MxCache, page_table, starts, tokens: int, dtype="bf16", k_out=None, v_out=None):
    """(k, v) [tokens, heads, dim]: the first tokens of every sequence, packed, in float32 or bfloat16, both exact
    (cfwd_mx_cache_read).

    ``page_table`` int32 [sequences, pages]; ``starts`` int32 [sequences + 1]: row starts[i] of the outputs is
    sequence i's token 0.  Rows behind starts[-1] are left as they were (undefined where the call allocates them).
    """
    torch = _torch()
    dev, sizes, parts = _check_cache(cache)
    sequences, pitch = _check_table(dev, page_table)
    _int32(dev, starts, (sequences + 1,), "starts")
    shape = (int(tokens), sizes[2], sizes[3])
    outs = []
    for out in (k_out, v_out):
        if out is None:
            code = _code(_MX_CODES, dtype, "dtype")
            if code == MXFP4:
                raise ValueError("dtype must be f32 or bf16")
            out = cache.k.codes.new_empty(shape, dtype=torch.float32 if code == F32 else torch.bfloat16)
        else:
            if out.shape != shape:
                raise ValueError("outputs must have the shape %s" % (shape,))
            _check_on(dev, out)
        outs.append(out)
    code = _float_code(outs[0])
    if outs[1].dtype != outs[0].dtype:
        raise ValueError("both outputs must have one dtype")
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return mx_cache_read(cache, page_table, starts, tokens, dtype, *outs)
    _check(_lib().cfwd_mx_cache_read(_mx_cache_read_desc(shape[0], sequences, pitch, code), parts, page_table.data_ptr(),
                                     starts.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(), _stream_of(dev)))
    return outs[0], outs[1]


def _workspace(workspace, need: int, like, dev: int):
    """(tensor, address, bytes) of the caller's workspace, or of a new one where one is needed, on ``like``'s GPU."""
    if workspace is not None:
        _check_on(dev, workspace)
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if not need:
        return None, None, 0
    workspace = like.new_empty((-(-need // like.element_size()),))
    return workspace, workspace.data_ptr(), need


@functools.lru_cache(maxsize=1024)
def _mx_cache_attention_desc(dev, cache_sizes, *sizes):
    """(descriptor reference, workspace bytes) on GPU ``dev``, the current one, whose CUs decide about the workspace."""
    desc, b = MxCacheAttentionDesc(*sizes), ctypes.c_size_t()
    _check(_lib().cfwd_mx_cache_attention_workspace_size(ctypes.byref(desc), ctypes.byref(MxCacheParts(*cache_sizes)),
                                                         ctypes.byref(b)))
    return ctypes.byref(desc), b.value


def mx_cache_attention(q, cache: MxCache, page_table, lengths, scale: Optional[float] = None, out=None, workspace=None):
    """softmax(scale q K^T) V over each sequence's cache (cfwd_mx_cache_attention).

    ``q`` bfloat16 [sequences, heads, dim], or [sequences, tokens, heads, dim]
    for several new tokens each: query i of them sees the first lengths - tokens + 1 + i
    tokens of its sequence.  ``page_table`` int32 [sequences, pages], ``lengths`` int32 [sequences]
    (the new tokens, which are in the cache already, among them).  ``scale``: default dim^-0.5.
    ``workspace`` (uint8, bytes as ``cfwd_mx_cache_attention_workspace_size`` says) is allocated when not given.
    """
    dev, sizes, parts = _check_cache(cache)
    if q.dim() not in (3, 4):
        raise ValueError("q must be [sequences, heads, dim] or [sequences, tokens, heads, dim]")
    shape, stride = q.shape, q.stride()
    sequences, tokens, heads = shape[0], shape[1] if len(shape) == 4 else 1, shape[-2]
    row = heads * shape[-1]  # the stride of an axis of one may be any number, and does not count
    seq_stride = stride[0] if sequences > 1 else tokens * row
    token_stride = stride[1] if tokens > 1 else row
    head_stride = stride[-2] if heads > 1 else shape[-1]
    if shape[-1] != sizes[3]:
        raise ValueError("q has heads of %d values, the cache of %d" % (shape[-1], sizes[3]))
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last axis of q must be dense")
    if q.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    rows, pitch = _check_table(dev, page_table)
    if rows != sequences:
        raise ValueError("page_table must have a row for each of %d sequences" % sequences)
    _int32(dev, lengths, (sequences,), "lengths")
    code = _float_code(q)
    if out is None:
        out = q.new_empty(tuple(shape))
    else:
        if out.shape != shape or out.dtype != q.dtype:
            raise ValueError("out must be as q")
        _check_on(dev, out)
    scale = float(scale) if scale is not None else shape[-1] ** -0.5
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return mx_cache_attention(q, cache, page_table, lengths, scale, out, workspace)
    desc, need = _mx_cache_attention_desc(dev, sizes, sequences, tokens, heads, pitch, scale, code, seq_stride,
                                          token_stride, head_stride)
    workspace, ws, ws_bytes = _workspace(workspace, need, q, dev)
    _check(_lib().cfwd_mx_cache_attention(desc, parts, q.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
                                          out.data_ptr(), ws, ws_bytes, _stream_of(dev)))
    return out


@functools.lru_cache(maxsize=1024)
def _attention_desc(dev, *sizes):
    """(descriptor reference, workspace bytes) on GPU ``dev``, the current one, whose CUs decide about the workspace."""
    desc, b = AttentionDesc(*sizes), ctypes.c_size_t()
    _check(_lib().cfwd_attention_workspace_size(ctypes.byref(desc), ctypes.byref(b)))
    return ctypes.byref(desc), b.value


def attention(q, k, v, q_starts, k_starts=None, causal: bool = True, scale: Optional[float] = None, out=None,
              workspace=None):
    """softmax(scale q k^T) v of packed prompts (cfwd_attention).

    ``q`` bfloat16 [tokens, heads, dim], ``k`` and ``v`` [key tokens, kv heads, dim] with dense dims; tokens and heads may
    be strided, as parts of one projection's output are.  Sequence i owns rows q_starts[i] .. q_starts[i + 1] - 1 of q and
    the same of k_starts (default: q_starts) of k and v; both int32 [sequences + 1].  ``causal``: a sequence's
    last query sees all its keys, the one before it one fewer, and so on; a query that sees none gives 0.  ``scale``:
    default dim^-0.5.  Rows of ``out`` behind the last sequence are left as they were (undefined where the call
    allocates it).  ``workspace`` (uint8, bytes as ``cfwd_attention_workspace_size`` says) is allocated when not given.
    """
    dev = q.get_device()
    tokens, heads, dim, qs, qh = _heads_of(q, "q")
    kt, kv_heads, kd, ks, kh = _heads_of(k, "k")
    vt, vheads, vd, vs, vh = _heads_of(v, "v")
    if kd != dim or (vt, vheads, vd) != (kt, kv_heads, kd) or not q.dtype == k.dtype == v.dtype:
        raise ValueError("q, k and v must have one dim and dtype, k and v one shape")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    if k_starts is None:
        k_starts = q_starts
    sequences = q_starts.numel() - 1
    if sequences < 0:
        raise ValueError("q_starts must be int32 [sequences + 1]")
    _int32(dev, q_starts, (sequences + 1,), "q_starts")
    _int32(dev, k_starts, (sequences + 1,), "k_starts")
    code = _float_code(q)
    if out is None:
        out = q.new_empty((tokens, heads, dim))
    else:
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must be as q")
        _check_on(dev, out)
    scale = float(scale) if scale is not None else dim ** -0.5
    guard = _guard(dev)
    if guard is not None:
        with guard:
            return attention(q, k, v, q_starts, k_starts, causal, scale, out, workspace)
    desc, need = _attention_desc(dev, tokens, kt, sequences, heads, kv_heads, dim, int(bool(causal)), scale, code, qs, qh,
                                 ks, kh, vs, vh)
    workspace, ws, ws_bytes = _workspace(workspace, need, q, dev)
    _check(_lib().cfwd_attention(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_starts.data_ptr(),
                                 k_starts.data_ptr(), out.data_ptr(), ws, ws_bytes, _stream_of(dev)))
    return out
