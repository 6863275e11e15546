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
