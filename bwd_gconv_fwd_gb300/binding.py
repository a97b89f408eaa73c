"""ctypes binding of libgconv.so (include/gconv.h): argument marshalling only.

Every function here forwards to the C entry point of the same name; all
arithmetic runs in the library's CUDA kernels.  There is no CPU fallback: if
libgconv.so is missing the first call raises.  PyTorch only supplies device
memory (tensors, workspaces) and the CUDA stream.

Geometry is the ABI's 14-tuple ``(N, C_in, H, W, C_out, kH, kW, stride, pad_top,
pad_bottom, pad_left, pad_right, dilation, groups)``, or the 16-tuple of the per-axis
entry points ``(N, C_in, H, W, C_out, kH, kW, stride_h, stride_w, pad_top, pad_bottom,
pad_left, pad_right, dilation_h, dilation_w, groups)`` (the ``gconv_geometry`` record);
the tensor-level wrappers derive it from the tensor shapes plus ``stride`` (an int or
(s_h, s_w)), ``padding`` (an int, (p_h, p_w) or (top, bottom, left, right)),
``dilation`` (an int or (d_h, d_w)) and ``groups``.  They call the 14-integer entry
points when the request fits them (equal strides and dilations, fp32 outputs, no fused
bias gradient) and the per-axis ``*_ex`` entry points otherwise.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgconv.so")

GCONV_OK, GCONV_ERR_INVALID_ARG, GCONV_ERR_UNSUPPORTED, GCONV_ERR_WORKSPACE, GCONV_ERR_CUDA, \
    GCONV_ERR_TIMEOUT = range(6)
GCONV_F32, GCONV_BF16 = 0, 1
PASS_FWD, PASS_BWD_DATA, PASS_BWD_WEIGHT, PASS_BWD_BIAS = range(4)
PATH_NONE, PATH_DIRECT, PATH_TC_IGEMM, PATH_TC_FC, PATH_REDUCE, PATH_TC_GEMM = range(6)
PATH_NAMES = {PATH_NONE: "none", PATH_DIRECT: "direct", PATH_TC_IGEMM: "tc_igemm",
              PATH_TC_FC: "tc_fc", PATH_REDUCE: "reduce", PATH_TC_GEMM: "tc_gemm1x1"}

EXPORTED = ("gconv_out_shape", "gconv_workspace_size", "gconv_plan", "gconv_fwd", "gconv_bwd_data",
            "gconv_bwd_weight", "gconv_bwd_bias", "gconv_check_device_error", "gconv_status_string",
            "gconv_debug_force_path", "gconv_debug_set_wait_limit", "gconv_debug_set_trace", "gconv_bwd_weight_noalloc",
            "gconv_noalloc_scratch_bytes", "gconv_step_host", "gconv_step_device_bytes",
            "gconv_out_shape_ex", "gconv_workspace_size_ex", "gconv_plan_ex", "gconv_fwd_ex", "gconv_bwd_data_ex",
            "gconv_bwd_weight_ex", "gconv_bwd_bias_ex", "gconv_step_workspace_size_ex", "gconv_step_plan_ex", "gconv_step_ex",
            "gconv_debug_set_step_events", "gconv_debug_set_wgrad_tma",
            "gconv_block_workspace_size", "gconv_norm_fwd", "gconv_norm_bwd", "gconv_join_fwd", "gconv_join_bwd",
            "gconv_orthogonalize_workspace_size", "gconv_orthogonalize", "gconv_muon_step",
            "gconv_causal_workspace_size", "gconv_causal_fwd", "gconv_causal_bwd",
            "gconv_scan_saved_size", "gconv_scan_workspace_size", "gconv_scan_fwd", "gconv_scan_bwd",
            "gconv_dropout_fwd", "gconv_dropout_bwd")

GATE_NONE, GATE_FULL, GATE_CHANNEL = range(3)
ACTS = {"none": 0, "sigmoid": 1, "silu": 2}


class Geometry(ctypes.Structure):
    """The gconv_geometry record of include/gconv.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("N", "C_in", "H", "W", "C_out", "kH", "kW", "stride_h", "stride_w",
                                             "pad_top", "pad_bottom", "pad_left", "pad_right", "dilation_h",
                                             "dilation_w", "groups")]


class Block(ctypes.Structure):
    """The gconv_block record of include/gconv.h."""
    _fields_ = [("N", ctypes.c_int), ("C", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
                ("groups", ctypes.c_int), ("eps", ctypes.c_float), ("gate", ctypes.c_int), ("act", ctypes.c_int)]


class Matrices(ctypes.Structure):
    """The gconv_matrices record of include/gconv.h."""
    _fields_ = [("count", ctypes.c_int), ("rows", ctypes.c_int), ("cols", ctypes.c_int)]


class Muon(ctypes.Structure):
    """The gconv_muon record of include/gconv.h."""
    _fields_ = [(n, ctypes.c_float) for n in ("lr", "beta", "weight_decay", "scale", "eps")] + \
        [("nesterov", ctypes.c_int), ("steps", ctypes.c_int), ("coeffs", ctypes.POINTER(ctypes.c_float))]


class Causal(ctypes.Structure):
    """The gconv_causal record of include/gconv.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("N", "C", "L", "taps", "act")] + \
        [(n, ctypes.c_longlong) for n in ("x_batch", "y_batch", "dy_batch", "dx_batch")]


class Scan(ctypes.Structure):
    """The gconv_scan record of include/gconv.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("N", "C", "L", "groups", "states", "softplus")] + \
        [(n + "_batch", ctypes.c_longlong) for n in ("u", "delta", "z", "B", "C", "y", "dy", "du", "ddelta", "dz", "dB", "dC")]


def per_axis(geom):
    """16-integer form of a 14- or 16-integer geometry."""
    g = tuple(int(v) for v in geom)
    if len(g) == 16:
        return g
    if len(g) != 14:
        raise ValueError("geometry must have 14 or 16 integers")
    N, Cin, H, W, Cout, kH, kW, s, pt, pb, pl, pr, d, G = g
    return (N, Cin, H, W, Cout, kH, kW, s, s, pt, pb, pl, pr, d, d, G)


def square(geom):
    """The 14-integer form when strides and dilations agree across axes, else None."""
    g = per_axis(geom)
    N, Cin, H, W, Cout, kH, kW, sh, sw, pt, pb, pl, pr, dh, dw, G = g
    if sh != sw or dh != dw:
        return None
    return (N, Cin, H, W, Cout, kH, kW, sh, pt, pb, pl, pr, dh, G)


def geometry_record(geom):
    return Geometry(*per_axis(geom))

_lib = None


class GconvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib():
    """Load libgconv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run bwd_gconv_fwd_gb300.build.build() "
                           "(or __graft_entry__.build()) -- there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    i, vp, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    geo = [i] * 14
    L.gconv_out_shape.argtypes = geo + [ctypes.POINTER(i), ctypes.POINTER(i)]
    L.gconv_out_shape.restype = i
    L.gconv_workspace_size.argtypes = geo + [i, i]
    L.gconv_workspace_size.restype = sz
    L.gconv_plan.argtypes = geo + [i, i, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.gconv_plan.restype = i
    L.gconv_fwd.argtypes = geo + [i, vp, vp, vp, vp, vp, sz, vp]
    L.gconv_fwd.restype = i
    L.gconv_bwd_data.argtypes = geo + [i, vp, vp, vp, vp, sz, vp]
    L.gconv_bwd_data.restype = i
    L.gconv_bwd_weight.argtypes = geo + [i, vp, vp, vp, vp, sz, vp]
    L.gconv_bwd_weight.restype = i
    L.gconv_bwd_bias.argtypes = geo + [i, vp, vp, vp, sz, vp]
    L.gconv_bwd_bias.restype = i
    L.gconv_bwd_weight_noalloc.argtypes = geo + [i, vp, vp, vp, vp]
    L.gconv_bwd_weight_noalloc.restype = i
    L.gconv_noalloc_scratch_bytes.argtypes = []
    L.gconv_noalloc_scratch_bytes.restype = sz
    L.gconv_step_host.argtypes = geo + [i, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.gconv_step_host.restype = i
    L.gconv_step_device_bytes.argtypes = geo + [i, i]
    L.gconv_step_device_bytes.restype = sz
    L.gconv_check_device_error.argtypes = [vp]
    L.gconv_check_device_error.restype = i
    L.gconv_status_string.argtypes = [i]
    L.gconv_status_string.restype = ctypes.c_char_p
    L.gconv_debug_force_path.argtypes = [i]
    L.gconv_debug_force_path.restype = None
    L.gconv_debug_set_wait_limit.argtypes = [ctypes.c_longlong]
    L.gconv_debug_set_wait_limit.restype = None
    L.gconv_debug_set_wgrad_tma.argtypes = [i]
    L.gconv_debug_set_wgrad_tma.restype = None
    L.gconv_debug_set_trace.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    L.gconv_debug_set_trace.restype = None
    gp = ctypes.POINTER(Geometry)
    L.gconv_out_shape_ex.argtypes = [gp, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.gconv_out_shape_ex.restype = i
    L.gconv_workspace_size_ex.argtypes = [gp, i, i]
    L.gconv_workspace_size_ex.restype = sz
    L.gconv_plan_ex.argtypes = [gp, i, i, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.gconv_plan_ex.restype = i
    L.gconv_fwd_ex.argtypes = [gp, i, i, vp, vp, vp, vp, vp, sz, vp]
    L.gconv_fwd_ex.restype = i
    L.gconv_bwd_data_ex.argtypes = [gp, i, i, vp, vp, vp, vp, sz, vp]
    L.gconv_bwd_data_ex.restype = i
    L.gconv_bwd_weight_ex.argtypes = [gp, i, vp, vp, vp, vp, vp, sz, vp]
    L.gconv_bwd_weight_ex.restype = i
    L.gconv_bwd_bias_ex.argtypes = [gp, i, vp, vp, vp, sz, vp]
    L.gconv_bwd_bias_ex.restype = i
    L.gconv_step_workspace_size_ex.argtypes = [gp, i]
    L.gconv_step_workspace_size_ex.restype = sz
    L.gconv_step_ex.argtypes = [gp, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.gconv_step_ex.restype = i
    L.gconv_step_plan_ex.argtypes = [gp, i, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.gconv_step_plan_ex.restype = i
    L.gconv_debug_set_step_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i]
    L.gconv_debug_set_step_events.restype = None
    bp = ctypes.POINTER(Block)
    L.gconv_block_workspace_size.argtypes = [bp, i]
    L.gconv_block_workspace_size.restype = sz
    L.gconv_norm_fwd.argtypes = [bp, i, vp, vp, vp, vp]
    L.gconv_norm_fwd.restype = i
    L.gconv_norm_bwd.argtypes = [bp, i, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.gconv_norm_bwd.restype = i
    L.gconv_join_fwd.argtypes = [bp, i] + [vp] * 9
    L.gconv_join_fwd.restype = i
    L.gconv_join_bwd.argtypes = [bp, i] + [vp] * 15 + [sz, vp]
    L.gconv_join_bwd.restype = i
    mp = ctypes.POINTER(Matrices)
    L.gconv_orthogonalize_workspace_size.argtypes = [mp]
    L.gconv_orthogonalize_workspace_size.restype = sz
    L.gconv_orthogonalize.argtypes = [mp, i, i, vp, vp, i, ctypes.POINTER(ctypes.c_float), ctypes.c_float, vp, sz, vp]
    L.gconv_orthogonalize.restype = i
    L.gconv_muon_step.argtypes = [mp, ctypes.POINTER(Muon)] + [vp] * 7 + [sz, vp]
    L.gconv_muon_step.restype = i
    cp, sp = ctypes.POINTER(Causal), ctypes.POINTER(Scan)
    L.gconv_causal_workspace_size.argtypes = [cp, i]
    L.gconv_causal_workspace_size.restype = sz
    L.gconv_causal_fwd.argtypes = [cp, i] + [vp] * 8
    L.gconv_causal_fwd.restype = i
    L.gconv_causal_bwd.argtypes = [cp, i] + [vp] * 12 + [sz, vp]
    L.gconv_causal_bwd.restype = i
    L.gconv_scan_saved_size.argtypes = [sp, i, i]
    L.gconv_scan_saved_size.restype = sz
    L.gconv_scan_workspace_size.argtypes = [sp, i, i]
    L.gconv_scan_workspace_size.restype = sz
    L.gconv_scan_fwd.argtypes = [sp, i] + [vp] * 14 + [sz, vp]
    L.gconv_scan_fwd.restype = i
    L.gconv_scan_bwd.argtypes = [sp, i] + [vp] * 22 + [sz, vp]
    L.gconv_scan_bwd.restype = i
    ll, db = ctypes.c_longlong, ctypes.c_double
    L.gconv_dropout_fwd.argtypes = [ll, i, vp, vp, vp, db, vp, vp]
    L.gconv_dropout_fwd.restype = i
    L.gconv_dropout_bwd.argtypes = [ll, i, vp, vp, db, vp, vp]
    L.gconv_dropout_bwd.restype = i
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().gconv_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != GCONV_OK:
        raise GconvError(status, what)


# ---- host-only queries ---------------------------------------------------------

def gconv_out_shape(geom):
    ho, wo = ctypes.c_int(), ctypes.c_int()
    if len(geom) == 16:
        rec = geometry_record(geom)
        _check(lib().gconv_out_shape_ex(ctypes.byref(rec), ctypes.byref(ho), ctypes.byref(wo)), "gconv_out_shape_ex")
    else:
        _check(lib().gconv_out_shape(*map(int, geom), ctypes.byref(ho), ctypes.byref(wo)), "gconv_out_shape")
    return ho.value, wo.value


def gconv_workspace_size(geom, dtype: int, pass_: int) -> int:
    if len(geom) == 16:
        rec = geometry_record(geom)
        n = lib().gconv_workspace_size_ex(ctypes.byref(rec), int(dtype), int(pass_))
    else:
        n = lib().gconv_workspace_size(*map(int, geom), int(dtype), int(pass_))
    if n == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_workspace_size")
    return int(n)


def gconv_plan(geom, dtype: int, pass_: int):
    """(path, launches) the library would use for this call."""
    path, launches = ctypes.c_int(), ctypes.c_int()
    if len(geom) == 16:
        rec = geometry_record(geom)
        _check(lib().gconv_plan_ex(ctypes.byref(rec), int(dtype), int(pass_), ctypes.byref(path),
                                   ctypes.byref(launches)), "gconv_plan_ex")
    else:
        _check(lib().gconv_plan(*map(int, geom), int(dtype), int(pass_), ctypes.byref(path),
                                ctypes.byref(launches)), "gconv_plan")
    return path.value, launches.value


def gconv_step_workspace_size(geom, dtype: int) -> int:
    """Workspace bytes gconv_step_ex needs for this geometry (14 or 16 integers)."""
    rec = geometry_record(per_axis(geom))
    n = lib().gconv_step_workspace_size_ex(ctypes.byref(rec), int(dtype))
    if n == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_step_workspace_size_ex")
    return int(n)


def gconv_step_plan(geom, dtype: int):
    """(shared, launches) of gconv_step_ex for this geometry: whether the passes share their
    blocked copies, and the step's kernel launches without db."""
    rec = geometry_record(per_axis(geom))
    shared, launches = ctypes.c_int(), ctypes.c_int()
    _check(lib().gconv_step_plan_ex(ctypes.byref(rec), int(dtype), ctypes.byref(shared), ctypes.byref(launches)),
           "gconv_step_plan_ex")
    return bool(shared.value), launches.value


def gconv_debug_force_path(path: int):
    lib().gconv_debug_force_path(int(path))


def gconv_debug_set_wait_limit(limit: int):
    lib().gconv_debug_set_wait_limit(int(limit))


def gconv_debug_set_wgrad_tma(enable: bool):
    """Test hook: False makes the tensor-core weight gradient stage its tiles by cp.async."""
    lib().gconv_debug_set_wgrad_tma(1 if enable else 0)



def gconv_debug_set_trace(device_ptr: int, nbytes: int):
    """Sets (or, with 0, clears) the device buffer the correlation kernel writes phase stamps to."""
    lib().gconv_debug_set_trace(ctypes.c_void_p(device_ptr or None), int(nbytes))


def gconv_debug_set_step_events(events):
    """Sets (a sequence of four torch.cuda.Event, each recorded once so that it exists) or,
    with None, clears the events gconv_step_ex records at its pass boundaries."""
    if not events:
        lib().gconv_debug_set_step_events(None, 0)
        return
    if len(events) != 4:
        raise ValueError("four events: start, after forward, after backward-data, after the weight gradient")
    arr = (ctypes.c_void_p * 4)(*(ctypes.c_void_p(e.cuda_event) for e in events))
    lib().gconv_debug_set_step_events(arr, 4)


def gconv_check_device_error(stream=None) -> int:
    """Synchronise the stream and return the status of the device error word."""
    return int(lib().gconv_check_device_error(_stream_ptr(stream)))


# ---- marshalling helpers -----------------------------------------------------

def _stream_ptr(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return GCONV_BF16
    if t == torch.float32:
        return GCONV_F32
    raise TypeError(f"unsupported input dtype {t}; use bfloat16 or float32")


def _pads(padding):
    if isinstance(padding, int):
        return (padding,) * 4
    p = tuple(int(v) for v in padding)
    if len(p) == 2:
        return (p[0], p[0], p[1], p[1])
    if len(p) != 4:
        raise ValueError("padding is an int, (ph, pw) or (top, bottom, left, right)")
    return p


def _pair(v):
    if isinstance(v, int):
        return int(v), int(v)
    a, b = (int(u) for u in v)
    return a, b


def geometry(x_shape, w_shape, stride=1, padding=0, dilation=1, groups=1):
    """The ABI geometry: a 14-tuple when strides and dilations agree across axes, else the
    16-tuple of the per-axis entry points."""
    N, Cin, H, W = (int(v) for v in x_shape)
    Cout, cgi, kH, kW = (int(v) for v in w_shape)
    if cgi * int(groups) != Cin:
        raise GconvError(GCONV_ERR_INVALID_ARG, f"weight has {cgi} input channels per group, "
                                                f"x has {Cin} channels for {groups} groups")
    pt, pb, pl, pr = _pads(padding)
    sh, sw = _pair(stride)
    dh, dw = _pair(dilation)
    if sh == sw and dh == dw:
        return (N, Cin, H, W, Cout, kH, kW, sh, pt, pb, pl, pr, dh, int(groups))
    return (N, Cin, H, W, Cout, kH, kW, sh, sw, pt, pb, pl, pr, dh, dw, int(groups))


def _dev(t: torch.Tensor, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _scratch(nbytes, device, stream):
    """A workspace tensor from the pool of the stream that the call's kernels run on: what the
    allocator hands out next with the same memory, and what had it before, are then ordered with them.
    The caller holds it until the kernels are launched."""
    if stream is not None:
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        if handle != torch.cuda.current_stream(device).cuda_stream:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
            with torch.cuda.stream(stream):
                return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(geom, dt, pass_, workspace, device, stream):
    """(tensor, pointer, bytes) of a pass's workspace."""
    need = gconv_workspace_size(geom, dt, pass_)
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = _scratch(need, device, stream)
    return workspace, ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()


# ---- the four passes (tensor level) -------------------------------------------

def _out_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GCONV_F32
    if t.dtype == torch.bfloat16:
        return GCONV_BF16
    raise TypeError(f"unsupported output dtype {t.dtype}; use float32 or bfloat16")


def gconv_fwd(x, w, bias, y, *, stride=1, padding=0, dilation=1, groups=1, workspace=None, stream=None):
    """y <- conv(x, w) + bias (bias may be None).  y: fp32 or bf16 [N, C_out, Ho, Wo]."""
    geom = geometry(x.shape, w.shape, stride, padding, dilation, groups)
    dt, odt = dtype_code(x.dtype), _out_code(y)
    held, ws, wsb = _workspace(geom, dt, PASS_FWD, workspace, x.device, stream)
    args = (_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _dev(y, "y"), ws, wsb, _stream_ptr(stream))
    if len(geom) == 14 and odt == GCONV_F32:
        _check(lib().gconv_fwd(*geom, dt, *args), "gconv_fwd")
    else:
        rec = geometry_record(geom)
        _check(lib().gconv_fwd_ex(ctypes.byref(rec), dt, odt, *args), "gconv_fwd_ex")
    return y


def gconv_bwd_data(dy, w, dx, *, stride=1, padding=0, dilation=1, groups=1, workspace=None, stream=None):
    """dx <- gradient of <y, dy> w.r.t. x.  dx: fp32 or bf16 [N, C_in, H, W]."""
    geom = geometry(dx.shape, w.shape, stride, padding, dilation, groups)
    dt, odt = dtype_code(dy.dtype), _out_code(dx)
    held, ws, wsb = _workspace(geom, dt, PASS_BWD_DATA, workspace, dy.device, stream)
    args = (_dev(dy, "dy"), _dev(w, "w"), _dev(dx, "dx"), ws, wsb, _stream_ptr(stream))
    if len(geom) == 14 and odt == GCONV_F32:
        _check(lib().gconv_bwd_data(*geom, dt, *args), "gconv_bwd_data")
    else:
        rec = geometry_record(geom)
        _check(lib().gconv_bwd_data_ex(ctypes.byref(rec), dt, odt, *args), "gconv_bwd_data_ex")
    return dx


def gconv_bwd_weight(x, dy, dw, *, db=None, stride=1, padding=0, dilation=1, groups=1, workspace=None,
                     stream=None):
    """dw <- gradient of <y, dy> w.r.t. w, fp32 [C_out, C_in/G, kH, kW]; with db (fp32
    [C_out]) also the bias gradient of the same dy, in the same call."""
    geom = geometry(x.shape, dw.shape, stride, padding, dilation, groups)
    dt = dtype_code(x.dtype)
    held, ws, wsb = _workspace(geom, dt, PASS_BWD_WEIGHT, workspace, x.device, stream)
    if len(geom) == 14 and db is None:
        _check(lib().gconv_bwd_weight(*geom, dt, _dev(x, "x"), _dev(dy, "dy"), _dev(dw, "dw"), ws, wsb,
                                      _stream_ptr(stream)), "gconv_bwd_weight")
    else:
        rec = geometry_record(geom)
        _check(lib().gconv_bwd_weight_ex(ctypes.byref(rec), dt, _dev(x, "x"), _dev(dy, "dy"), _dev(dw, "dw"),
                                         _dev(db, "db"), ws, wsb, _stream_ptr(stream)), "gconv_bwd_weight_ex")
    return dw


def gconv_bwd_weight_noalloc(x, dy, dw, *, stride=1, padding=0, dilation=1, groups=1, stream=None):
    """dw <- gradient w.r.t. w, using the library's fixed scratch instead of a workspace
    (for callers that cannot allocate device memory; see include/gconv.h)."""
    geom = geometry(x.shape, dw.shape, stride, padding, dilation, groups)
    dt = dtype_code(x.dtype)
    _check(lib().gconv_bwd_weight_noalloc(*geom, dt, _dev(x, "x"), _dev(dy, "dy"), _dev(dw, "dw"),
                                          _stream_ptr(stream)), "gconv_bwd_weight_noalloc")
    return dw


def gconv_noalloc_scratch_bytes() -> int:
    return int(lib().gconv_noalloc_scratch_bytes())


def gconv_step_device_bytes(geom, dtype: int, with_bias: bool = True) -> int:
    n = lib().gconv_step_device_bytes(*map(int, geom), int(dtype), int(bool(with_bias)))
    if n == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_step_device_bytes")
    return int(n)


def _host(t, name: str):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host tensor")
    return ctypes.c_void_p(t.data_ptr())


def gconv_step(x, w, bias, dy, y, dx, dw, db=None, *, stride=1, padding=0, dilation=1, groups=1, workspace=None,
               stream=None):
    """One step on device tensors: y <- forward(x, w, bias), dx <- backward-data(dy, w),
    dw <- weight gradient(x, dy) and, with db, the bias gradient; y and dx fp32 or bf16
    (the same dtype), dw and db fp32.  Equal bit for bit to the separate passes."""
    geom = per_axis(geometry(x.shape, w.shape, stride, padding, dilation, groups))
    dt, odt = dtype_code(x.dtype), _out_code(y)
    if _out_code(dx) != odt:
        raise TypeError("y and dx must have the same dtype")
    need = gconv_step_workspace_size(geom, dt)
    if need and workspace is None:
        workspace = _scratch(need, x.device, stream)
    ws = ctypes.c_void_p(workspace.data_ptr()) if need else None
    wsb = workspace.numel() * workspace.element_size() if need else 0
    rec = geometry_record(geom)
    _check(lib().gconv_step_ex(ctypes.byref(rec), dt, odt, _dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"),
                               _dev(dy, "dy"), _dev(y, "y"), _dev(dx, "dx"), _dev(dw, "dw"), _dev(db, "db"), ws, wsb,
                               _stream_ptr(stream)), "gconv_step_ex")
    return y, dx, dw, db


def gconv_step_host(x, w, bias, dy, y, dx, dw, db, device_buffer, *, stride=1, padding=0, dilation=1,
                    groups=1, stream=None):
    """One step on host tensors (pinned for overlap): inputs copied in, the four passes,
    y/dx/dw/db copied back; done when `stream` reaches this point (see include/gconv.h)."""
    geom = geometry(x.shape, w.shape, stride, padding, dilation, groups)
    dt = dtype_code(x.dtype)
    if not device_buffer.is_cuda:
        raise ValueError("device_buffer must be a device tensor")
    _check(lib().gconv_step_host(*geom, dt, _host(x, "x"), _host(w, "w"), _host(bias, "bias"), _host(dy, "dy"),
                                 _host(y, "y"), _host(dx, "dx"), _host(dw, "dw"), _host(db, "db"),
                                 ctypes.c_void_p(device_buffer.data_ptr()),
                                 device_buffer.numel() * device_buffer.element_size(), _stream_ptr(stream)),
           "gconv_step_host")


def gconv_step_host_ptr(geom, dt, x, w, bias, dy, y, dx, dw, db, buf, buf_bytes, stream=0):
    """Pointer-level form of gconv_step_host (host pointers for tensors, a device buffer)."""
    _check(lib().gconv_step_host(*map(int, geom), int(dt), x, w, bias or None, dy, y, dx, dw, db, buf,
                                 int(buf_bytes), stream or None), "gconv_step_host")


def gconv_bwd_bias(dy, db, *, geom=None, workspace=None, stream=None):
    """db <- sum of dy over (N, Ho, Wo).  geom defaults to a 1x1 geometry on dy's shape."""
    if geom is None:
        N, C, Ho, Wo = (int(v) for v in dy.shape)
        geom = (N, C, Ho, Wo, C, 1, 1, 1, 0, 0, 0, 0, 1, 1)
    dt = dtype_code(dy.dtype)
    held, ws, wsb = _workspace(geom, dt, PASS_BWD_BIAS, workspace, dy.device, stream)
    if len(geom) == 14:
        _check(lib().gconv_bwd_bias(*geom, dt, _dev(dy, "dy"), _dev(db, "db"), ws, wsb, _stream_ptr(stream)),
               "gconv_bwd_bias")
    else:
        rec = geometry_record(geom)
        _check(lib().gconv_bwd_bias_ex(ctypes.byref(rec), dt, _dev(dy, "dy"), _dev(db, "db"), ws, wsb,
                                       _stream_ptr(stream)), "gconv_bwd_bias_ex")
    return db


# ---- block norm and block join ---------------------------------------------------
#
# These calls take microseconds on the GPU for small layers, so their marshalling is lean: a
# tensor's checks are five attribute reads, pointers pass as integers, and the records and
# workspace sizes, which depend on the sizes and the device's number of SMs, are made once for each set
# of sizes and device.

def _device_index():
    """The current device: part of what is kept for a set of sizes."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -1


def _like(t, shape, dtype, name):
    """Address of a contiguous CUDA tensor of this shape and dtype (0 for None)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must have shape {tuple(shape)} and dtype {dtype}")
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.data_ptr()


def _raw_stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


@functools.lru_cache(maxsize=1024)
def _block_record(N, C, H, W, groups, eps, gate, act, dt, device):
    """(record, its reference, workspace bytes of the backward calls, [C])."""
    if act not in ACTS:
        raise ValueError(f"act is one of {sorted(ACTS)}")
    block = Block(N, C, H, W, groups, eps, gate, ACTS[act])
    need = lib().gconv_block_workspace_size(ctypes.byref(block), dt)
    if need == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_block_workspace_size")
    return block, ctypes.byref(block), int(need), torch.Size((C,))


def _block(x, name, groups, eps, gate=None, act="none"):
    shape, dtype = x.shape, x.dtype
    if len(shape) != 4:
        raise ValueError(f"{name} is [N, C, H, W]")
    kind = GATE_NONE
    if gate is not None:
        kind = GATE_FULL if gate.shape == shape else GATE_CHANNEL
        if kind == GATE_CHANNEL and gate.shape != shape[:2]:
            raise ValueError("gate is [N, C, H, W] or [N, C]")
    dt = GCONV_BF16 if dtype is torch.bfloat16 else dtype_code(dtype)
    record = _block_record(*shape, int(groups), float(eps), kind, act, dt, x.get_device())
    return shape, dtype, dt, kind, *record


def _block_workspace(need, workspace, device, stream):
    if workspace is None:
        workspace = _scratch(need, device, stream)
    elif not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gconv_block_workspace_size(x_shape, dtype: int, groups: int = 1) -> int:
    """Workspace bytes gconv_norm_bwd and gconv_join_bwd need for activations of this shape."""
    N, C, H, W = (int(v) for v in x_shape)
    return _block_record(N, C, H, W, int(groups), 0.0, GATE_NONE, "none", int(dtype), _device_index())[2]


def gconv_norm_fwd(x, weight, y, *, groups=1, eps=1e-6, stream=None):
    """y <- x / rms(x over each group's channels) * weight, at every position (weight: fp32 [C]
    or None)."""
    s, d, dt, _, _, ref, _, c = _block(x, "x", groups, eps)
    st = lib().gconv_norm_fwd(ref, dt, _like(x, s, d, "x"), _like(weight, c, torch.float32, "weight"),
                              _like(y, s, d, "y"), _raw_stream(stream))
    if st:
        _check(st, "gconv_norm_fwd")
    return y


def gconv_norm_bwd(x, weight, dy, dx, dweight=None, *, dres=None, groups=1, eps=1e-6, workspace=None, stream=None):
    """dx <- dres + gradient of the norm w.r.t. x; dweight (fp32 [C]) <- gradient w.r.t. weight."""
    s, d, dt, _, _, ref, need, c = _block(x, "x", groups, eps)
    f = torch.float32
    ws, wp, wb = _block_workspace(need, workspace, x.device, stream)
    st = lib().gconv_norm_bwd(ref, dt, _like(x, s, d, "x"), _like(weight, c, f, "weight"), _like(dy, s, d, "dy"),
                              _like(dres, s, d, "dres"), _like(dx, s, d, "dx"), _like(dweight, c, f, "dweight"), wp, wb,
                              _raw_stream(stream))
    if st:
        _check(st, "gconv_norm_bwd")
    return dx, dweight


def gconv_join_fwd(res, h, out, *, gate=None, act="none", weight=None, scale=None, next=None, next_weight=None, groups=1,
                   eps=1e-6, stream=None):
    """out <- res + scale * act(gate) * (h / rms(h) * weight) and, with next, next <- out / rms(out) *
    next_weight.  gate: None, [N, C, H, W] or [N, C]; weight, scale, next_weight: fp32 [C] or None."""
    s, d, dt, kind, _, ref, _, c = _block(res, "res", groups, eps, gate, act)
    f = torch.float32
    st = lib().gconv_join_fwd(ref, dt, _like(res, s, d, "res"), _like(h, s, d, "h"),
                              _like(gate, s if kind != GATE_CHANNEL else s[:2], d, "gate"), _like(weight, c, f, "weight"),
                              _like(scale, c, f, "scale"), _like(next_weight, c, f, "next_weight"),
                              _like(out, s, d, "out"), _like(next, s, d, "next"), _raw_stream(stream))
    if st:
        _check(st, "gconv_join_fwd")
    return out, next


def gconv_join_bwd(h, dout, dh, *, gate=None, act="none", weight=None, scale=None, dgate=None, dweight=None, dscale=None,
                   out=None, next_weight=None, dnext=None, dres=None, dnext_weight=None, groups=1, eps=1e-6,
                   workspace=None, stream=None):
    """Gradients of gconv_join_fwd.  Without dnext (the join had no next) dout is the gradient of
    out; with it dres <- the whole gradient of out.  dgate: like gate for a full gate, fp32 [N, C]
    for a channel gate; dweight, dscale, dnext_weight: fp32 [C] or None."""
    s, d, dt, kind, _, ref, need, c = _block(h, "h", groups, eps, gate, act)
    f = torch.float32
    by_channel = kind == GATE_CHANNEL
    nc = s[:2] if by_channel else s
    ws, wp, wb = _block_workspace(need, workspace, h.device, stream)
    st = lib().gconv_join_bwd(ref, dt, _like(out, s, d, "out"), _like(h, s, d, "h"), _like(gate, nc, d, "gate"),
                              _like(weight, c, f, "weight"), _like(scale, c, f, "scale"),
                              _like(next_weight, c, f, "next_weight"), _like(dout, s, d, "dout"),
                              _like(dnext, s, d, "dnext"), _like(dres, s, d, "dres"), _like(dh, s, d, "dh"),
                              _like(dgate, nc, f if by_channel else d, "dgate"), _like(dweight, c, f, "dweight"),
                              _like(dscale, c, f, "dscale"), _like(dnext_weight, c, f, "dnext_weight"), wp, wb,
                              _raw_stream(stream))
    if st:
        _check(st, "gconv_join_bwd")
    return dh, dres


# ---- orthogonalised updates ------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _matrices(shape, groups, device):
    """(record, its reference, workspace bytes) of a weight shape."""
    if len(shape) < 2 or groups < 1 or shape[0] % groups:
        raise GconvError(GCONV_ERR_INVALID_ARG, f"{tuple(shape)} is not {groups} groups of matrices")
    cols = 1
    for v in shape[1:]:
        cols *= int(v)
    m = Matrices(groups, shape[0] // groups, cols)
    need = lib().gconv_orthogonalize_workspace_size(ctypes.byref(m))
    if need == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_orthogonalize_workspace_size")
    return m, ctypes.byref(m), int(need)


@functools.lru_cache(maxsize=64)
def _coeff_array(coeffs, steps):
    flat = [float(v) for t in coeffs for v in (t if isinstance(t, tuple) else (t,))]
    if len(flat) == 3:
        flat = flat * steps
    if len(flat) != 3 * steps:
        raise ValueError("coeffs is (a, b, c) or one such triple a step")
    return (ctypes.c_float * len(flat))(*flat)


def _coeffs(coeffs, steps):
    """(a, b, c) for every step, or one triple a step, as a float array (None: the library's)."""
    if coeffs is None:
        return None
    return _coeff_array(tuple(tuple(c) if hasattr(c, "__len__") else c for c in coeffs), int(steps))


def _orth_workspace(need, workspace, device, stream):
    if workspace is None:
        if need == 0:
            return None, 0, 0
        workspace = _scratch(need, device, stream)
    elif not (workspace.device == device and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor, on the device of the others")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gconv_orthogonalize_workspace_size(w_shape, groups: int = 1) -> int:
    """Workspace bytes of gconv_orthogonalize and gconv_muon_step for weights of this shape."""
    return _matrices(torch.Size(w_shape), int(groups), _device_index())[2]


def gconv_orthogonalize(g, out, *, groups=1, steps=5, coeffs=None, eps=1e-7, workspace=None, stream=None):
    """out <- each group's matrix of g ([C_out, ...]: C_out/groups rows) orthogonalised by `steps`
    Newton-Schulz steps.  g, out: fp32 or bf16; coeffs: (a, b, c), or one triple a step."""
    shape = g.shape
    dt, odt = dtype_code(g.dtype), _out_code(out)
    _, ref, need = _matrices(shape, int(groups), g.get_device())
    c = _coeffs(coeffs, steps)
    ws, wp, wb = _orth_workspace(need, workspace, g.device, stream)
    st = lib().gconv_orthogonalize(ref, dt, odt, _like(g, shape, g.dtype, "g"), _like(out, shape, out.dtype, "out"),
                                   int(steps), c, float(eps), wp, wb, _raw_stream(stream))
    if st:
        _check(st, "gconv_orthogonalize")
    return out


def gconv_muon_step(w, grad, momentum, *, w_out=None, m_out=None, w_bf16=None, groups=1, lr=0.02, beta=0.95,
                    weight_decay=0.0, scale=0.0, nesterov=True, steps=5, coeffs=None, eps=1e-7, workspace=None,
                    stream=None):
    """One Muon step: fp32 w and momentum are updated (in place unless w_out, m_out are given) from
    the fp32 weight gradient; w_bf16, when given, gets the new weights rounded to bf16."""
    w_out, m_out = w if w_out is None else w_out, momentum if m_out is None else m_out
    shape, f = w.shape, torch.float32
    _, ref, need = _matrices(shape, int(groups), w.get_device())
    opt = Muon(lr, beta, weight_decay, scale, eps, 1 if nesterov else 0, steps, _coeffs(coeffs, steps))
    ws, wp, wb = _orth_workspace(need, workspace, w.device, stream)
    st = lib().gconv_muon_step(ref, ctypes.byref(opt), _like(w, shape, f, "w"), _like(grad, shape, f, "grad"),
                               _like(momentum, shape, f, "momentum"), _like(w_out, shape, f, "w_out"),
                               _like(m_out, shape, f, "m_out"), _like(w_bf16, shape, torch.bfloat16, "w_bf16"), wp, wb,
                               _raw_stream(stream))
    if st:
        _check(st, "gconv_muon_step")
    return w_out, m_out


# ---- sequences: causal convolution and selective scan ------------------------------
#
# Activations are [N, C, L], or [N, C, H, W] and [N, C] with L = H W and 1: what follows the channels is one run of
# positions.  A tensor may be a slice of the channels of a larger one (whole sequences, further apart).

def _positions(shape):
    if len(shape) == 3:
        return shape[2]
    if len(shape) < 2:
        raise ValueError("activations are [N, C, ...]")
    count = 1
    for v in shape[2:]:
        count *= v
    return count


def _sequences(t, shape, dtype, device, name):
    """(address, elements between sequences or 0 for dense) of an activation tensor; (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} and dtype {dtype}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be a CUDA tensor, on the device of the others")
    if t.is_contiguous():
        return t.data_ptr(), 0
    if t.stride(0) <= 0 or not t[0].is_contiguous():
        raise ValueError(f"{name} must have contiguous sequences")
    return t.data_ptr(), t.stride(0)


def _array(t, shape, dtype, device, name):
    """Address of a contiguous tensor of this shape and dtype on the device (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} and dtype {dtype}")
    if t.get_device() != device or device < 0 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor, on the device of the others")
    return t.data_ptr()


def _lengths(lengths, n, device):
    return 0 if lengths is None else _array(lengths, torch.Size((n,)), torch.int32, device, "lengths")


def _stream_on(stream, device):
    """The stream's handle; the tensors have to be on the current device, which the kernels run on.  Asked for before the records
    below, whose sizes are the current device's."""
    now = torch._C._cuda_getDevice()
    if now != device:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{now}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(now)
    return stream if isinstance(stream, int) else stream.cuda_stream


@functools.lru_cache(maxsize=1024)
def _causal_record(shape, w_shape, act, strides, dt, device):
    """(record, its reference, workspace bytes of the gradient, [C], [N, C, K-1])."""
    if len(w_shape) not in (2, 4) or w_shape[0] != shape[1] or w_shape.numel() != shape[1] * w_shape[-1]:
        raise ValueError("w is [C, K] or [C, 1, 1, K]")
    if act not in ACTS:
        raise ValueError(f"act is one of {sorted(ACTS)}")
    N, C, L, taps = shape[0], shape[1], _positions(shape), w_shape[-1]
    rec = Causal(N, C, L, taps, ACTS[act], *strides)
    need = lib().gconv_causal_workspace_size(ctypes.byref(rec), dt)
    if need == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_causal_workspace_size")
    return rec, ctypes.byref(rec), int(need), torch.Size((C,)), torch.Size((N, C, taps - 1))


def gconv_causal_workspace_size(x_shape, taps: int, dtype: int) -> int:
    """Workspace bytes gconv_causal_bwd needs for activations of this shape."""
    return _causal_record(torch.Size(x_shape), torch.Size((x_shape[1], taps)), "none", (0, 0, 0, 0), int(dtype), _device_index())[2]


def gconv_causal_fwd(x, w, bias, y, *, act="none", state=None, state_out=None, lengths=None, stream=None):
    """y[t] <- act(bias + sum_k w[k] x[t - K + 1 + k]) for every channel; w: fp32 [C, K], bias: fp32 [C] or
    None, act: "none" or "silu".  state [N, C, K-1] holds the positions before the first (None: zeros), state_out, which
    may be state, gets the last ones.  lengths: int32 [N] or None; results behind a sequence's length are zero."""
    s, d, ws, f, dev = x.shape, x.dtype, w.shape, torch.float32, x.get_device()
    dt = GCONV_BF16 if d is torch.bfloat16 else dtype_code(d)
    (xp, xs), (yp, ys) = _sequences(x, s, d, dev, "x"), _sequences(y, s, d, dev, "y")
    on = _stream_on(stream, dev)
    _, ref, _, c, held = _causal_record(s, ws, act, (xs, ys, 0, 0), dt, dev)
    st = lib().gconv_causal_fwd(ref, dt, xp, _array(w, ws, f, dev, "w"), _array(bias, c, f, dev, "bias"), _array(state, held, d, dev, "state"),
                                _lengths(lengths, s[0], dev), yp, _array(state_out, held, d, dev, "state_out"), on)
    if st:
        _check(st, "gconv_causal_fwd")
    return y


def gconv_causal_bwd(x, w, bias, dy, dx, dw, dbias=None, *, act="none", state=None, lengths=None, dstate_out=None, dstate=None,
                     workspace=None, stream=None):
    """Gradients of gconv_causal_fwd: dx like x, dw and dbias fp32; dstate gets the gradient of state, dstate_out is that of
    state_out (None: none)."""
    s, d, ws, f, dev = x.shape, x.dtype, w.shape, torch.float32, x.get_device()
    dt = GCONV_BF16 if d is torch.bfloat16 else dtype_code(d)
    (xp, xs), (yp, ys), (dp, ds) = _sequences(x, s, d, dev, "x"), _sequences(dy, s, d, dev, "dy"), _sequences(dx, s, d, dev, "dx")
    on = _stream_on(stream, dev)
    _, ref, need, c, held = _causal_record(s, ws, act, (xs, 0, ys, ds), dt, dev)
    hold, sp, sb = _orth_workspace(need, workspace, x.device, stream)
    st = lib().gconv_causal_bwd(ref, dt, xp, _array(w, ws, f, dev, "w"), _array(bias, c, f, dev, "bias"), _array(state, held, d, dev, "state"),
                                _lengths(lengths, s[0], dev), yp, _array(dstate_out, held, d, dev, "dstate_out"), dp, _array(dw, ws, f, dev, "dw"),
                                _array(dbias, c, f, dev, "dbias"), _array(dstate, held, d, dev, "dstate"), sp, sb, on)
    if st:
        _check(st, "gconv_causal_bwd")
    return dx, dw, dbias


@functools.lru_cache(maxsize=1024)
def _scan_record(shape, B_shape, states, groups, softplus, strides, dt, device):
    """(record, its reference, workspace bytes forward and backward, bytes saved without and with a gate, [C], [C, states],
    [N, C, states])."""
    N, C, L = shape[0], shape[1], _positions(shape)
    if B_shape[:2] == (N, groups * states):
        own = B_shape[2:]
    elif B_shape[:3] == (N, groups, states):
        own = B_shape[3:]
    else:
        raise ValueError("B and C are [N, groups * states, ...] or [N, groups, states, ...] with A [C, states]")
    if torch.Size(own).numel() != L:
        raise ValueError("B and C have the positions of u")
    rec = Scan(N, C, L, groups, states, softplus, *strides)
    ref = ctypes.byref(rec)
    need = [lib().gconv_scan_workspace_size(ref, dt, back) for back in (0, 1)] + \
        [lib().gconv_scan_saved_size(ref, dt, gated) for gated in (0, 1)]
    if ctypes.c_size_t(-1).value in need:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_scan_workspace_size")
    return rec, ref, *map(int, need), torch.Size((C,)), torch.Size((C, states)), torch.Size((N, C, states))


def gconv_scan_saved_size(x_shape, states: int, dtype: int, gated: bool = False) -> int:
    """Bytes of what gconv_scan_fwd keeps for gconv_scan_bwd."""
    rec = Scan(int(x_shape[0]), int(x_shape[1]), _positions(x_shape), 1, int(states), 0)
    n = lib().gconv_scan_saved_size(ctypes.byref(rec), int(dtype), 1 if gated else 0)
    if n == ctypes.c_size_t(-1).value:
        raise GconvError(GCONV_ERR_INVALID_ARG, "gconv_scan_saved_size")
    return int(n)


def gconv_scan_workspace_size(x_shape, states: int, dtype: int, groups: int = 1, backward: bool = False) -> int:
    """Workspace bytes of gconv_scan_fwd or gconv_scan_bwd for activations of this shape."""
    s = torch.Size(x_shape)
    B = torch.Size((s[0], groups * states, _positions(s)))
    return _scan_record(s, B, int(states), int(groups), 0, (0,) * 12, int(dtype), _device_index())[3 if backward else 2]


def _scan_saved(saved, need, dev):
    if saved.get_device() != dev or not saved.is_contiguous() or saved.numel() * saved.element_size() < need:
        raise ValueError(f"saved is a contiguous CUDA tensor of at least {need} bytes (gconv_scan_saved_size)")
    return saved.data_ptr()


def gconv_scan_fwd(u, delta, A, B, C, y, *, D=None, z=None, delta_bias=None, softplus=True, groups=1, state=None,
                   state_out=None, lengths=None, saved=None, workspace=None, stream=None):
    """The selective scan: with d = softplus(delta + delta_bias), h[t] = exp(d A) h[t-1] + d B[t] u[t] and
    y <- (sum over the states of C[t] h[t] + D u) silu(z).  A: fp32 [C, states]; B, C: [N, groups * states, positions]
    or [N, groups, states, positions]; D, delta_bias: fp32 [C]; state, state_out (which may be state): fp32 [N, C, states]; lengths: int32 [N].
    saved (gconv_scan_saved_size bytes) keeps what gconv_scan_bwd needs."""
    s, d, bs, f, dev = u.shape, u.dtype, B.shape, torch.float32, u.get_device()
    dt = GCONV_BF16 if d is torch.bfloat16 else dtype_code(d)
    up, us = _sequences(u, s, d, dev, "u")
    dp, ds = _sequences(delta, s, d, dev, "delta")
    zp, zs = _sequences(z, s, d, dev, "z")
    yp, ys = _sequences(y, s, d, dev, "y")
    Bp, Bs = _sequences(B, bs, d, dev, "B")
    Cp, Cs = _sequences(C, bs, d, dev, "C")
    on = _stream_on(stream, dev)
    _, ref, need, _, plain, gated, c, cs, full = _scan_record(s, bs, A.shape[-1], int(groups), 1 if softplus else 0,
                                                              (us, ds, zs, Bs, Cs, ys, 0, 0, 0, 0, 0, 0), dt, dev)
    hold, wp, wb = _orth_workspace(need, workspace, u.device, stream)
    st = lib().gconv_scan_fwd(ref, dt, up, dp, _array(A, cs, f, dev, "A"), Bp, Cp, _array(D, c, f, dev, "D"), zp,
                              _array(delta_bias, c, f, dev, "delta_bias"), _array(state, full, f, dev, "state"), _lengths(lengths, s[0], dev), yp,
                              _array(state_out, full, f, dev, "state_out"),
                              0 if saved is None else _scan_saved(saved, plain if z is None else gated, dev), wp, wb, on)
    if st:
        _check(st, "gconv_scan_fwd")
    return y


def gconv_scan_bwd(u, delta, A, B, C, dy, saved, du, ddelta, dA, dB, dC, *, D=None, z=None, delta_bias=None, softplus=True,
                   groups=1, lengths=None, dD=None, dz=None, ddelta_bias=None, dstate_out=None, dstate=None, workspace=None,
                   stream=None):
    """Gradients of gconv_scan_fwd from its inputs and what it saved.  du, ddelta, dz like u, dB and dC like B; dA, dD,
    ddelta_bias fp32; dstate (fp32) gets the gradient of state, dstate_out is that of state_out (None: none)."""
    s, d, bs, f, dev = u.shape, u.dtype, B.shape, torch.float32, u.get_device()
    dt = GCONV_BF16 if d is torch.bfloat16 else dtype_code(d)
    t = [_sequences(v, shape, d, dev, name) for name, v, shape in
         (("u", u, s), ("delta", delta, s), ("z", z, s), ("B", B, bs), ("C", C, bs), ("dy", dy, s), ("du", du, s),
          ("ddelta", ddelta, s), ("dz", dz, s), ("dB", dB, bs), ("dC", dC, bs))]
    (up, us), (dp, ds), (zp, zs), (Bp, Bs), (Cp, Cs), (gp, gs), (dup, dus), (ddp, dds), (dzp, dzs), (dBp, dBs), (dCp, dCs) = t
    on = _stream_on(stream, dev)
    _, ref, _, need, plain, gated, c, cs, full = _scan_record(s, bs, A.shape[-1], int(groups), 1 if softplus else 0,
                                                              (us, ds, zs, Bs, Cs, 0, gs, dus, dds, dzs, dBs, dCs), dt,
                                                              dev)
    hold, wp, wb = _orth_workspace(need, workspace, u.device, stream)
    st = lib().gconv_scan_bwd(ref, dt, up, dp, _array(A, cs, f, dev, "A"), Bp, Cp, _array(D, c, f, dev, "D"), zp,
                              _array(delta_bias, c, f, dev, "delta_bias"), _lengths(lengths, s[0], dev),
                              _scan_saved(saved, plain if z is None else gated, dev), gp, _array(dstate_out, full, f, dev, "dstate_out"), dup,
                              ddp, _array(dA, cs, f, dev, "dA"), dBp, dCp, _array(dD, c, f, dev, "dD"), dzp,
                              _array(ddelta_bias, c, f, dev, "ddelta_bias"), _array(dstate, full, f, dev, "dstate"), wp, wb, on)
    if st:
        _check(st, "gconv_scan_bwd")
    return du, ddelta


# ---- dropout -----------------------------------------------------------------------

def _rng(rng, dev):
    return _array(rng, torch.Size((2,)), torch.int64, dev, "rng")


def gconv_dropout_fwd(x, y, rng, p, *, res=None, stream=None):
    """y <- x / (1 - p) where kept, else 0, plus res.  rng: int64 CUDA tensor (seed, step), which the mask follows from;
    use another pair for every tensor and step, and the same for the gradient.  y may be x or res."""
    s, d, dev = x.shape, x.dtype, x.get_device()
    st = lib().gconv_dropout_fwd(x.numel(), dtype_code(d), _array(x, s, d, dev, "x"), _array(res, s, d, dev, "res"), _rng(rng, dev), p,
                                 _array(y, s, d, dev, "y"), _stream_on(stream, dev))
    if st:
        _check(st, "gconv_dropout_fwd")
    return y


def gconv_dropout_bwd(dy, dx, rng, p, *, stream=None):
    """dx <- dy / (1 - p) where the forward call with this rng kept the element, else 0 (the gradient of res is dy)."""
    s, d, dev = dy.shape, dy.dtype, dy.get_device()
    st = lib().gconv_dropout_bwd(dy.numel(), dtype_code(d), _array(dy, s, d, dev, "dy"), _rng(rng, dev), p, _array(dx, s, d, dev, "dx"),
                                 _stream_on(stream, dev))
    if st:
        _check(st, "gconv_dropout_bwd")
    return dx


# ---- raw pointer level (same C signatures), for callers holding pointers ------

def gconv_fwd_ptr(geom, dt, x, w, bias, y, ws=0, ws_bytes=0, stream=0):
    _check(lib().gconv_fwd(*map(int, geom), int(dt), x, w, bias or None, y, ws or None, int(ws_bytes),
                           stream or None), "gconv_fwd")


def gconv_bwd_data_ptr(geom, dt, dy, w, dx, ws=0, ws_bytes=0, stream=0):
    _check(lib().gconv_bwd_data(*map(int, geom), int(dt), dy, w, dx, ws or None, int(ws_bytes),
                                stream or None), "gconv_bwd_data")


def gconv_bwd_weight_ptr(geom, dt, x, dy, dw, ws=0, ws_bytes=0, stream=0):
    _check(lib().gconv_bwd_weight(*map(int, geom), int(dt), x, dy, dw, ws or None, int(ws_bytes),
                                  stream or None), "gconv_bwd_weight")


def gconv_bwd_bias_ptr(geom, dt, dy, db, ws=0, ws_bytes=0, stream=0):
    _check(lib().gconv_bwd_bias(*map(int, geom), int(dt), dy, db, ws or None, int(ws_bytes),
                                stream or None), "gconv_bwd_bias")


# ---- per-axis entry points at pointer level (16-integer geometry) ------------

def gconv_fwd_ex_ptr(geom, dt, out_dt, x, w, bias, y, ws=0, ws_bytes=0, stream=0):
    rec = geometry_record(geom)
    _check(lib().gconv_fwd_ex(ctypes.byref(rec), int(dt), int(out_dt), x, w, bias or None, y, ws or None,
                              int(ws_bytes), stream or None), "gconv_fwd_ex")


def gconv_bwd_data_ex_ptr(geom, dt, out_dt, dy, w, dx, ws=0, ws_bytes=0, stream=0):
    rec = geometry_record(geom)
    _check(lib().gconv_bwd_data_ex(ctypes.byref(rec), int(dt), int(out_dt), dy, w, dx, ws or None, int(ws_bytes),
                                   stream or None), "gconv_bwd_data_ex")


def gconv_step_ex_ptr(geom, dt, out_dt, x, w, bias, dy, y, dx, dw, db=0, ws=0, ws_bytes=0, stream=0):
    """Pointer-level gconv_step_ex: y, dx, dw and (db not 0) db of one layer in one call."""
    rec = geometry_record(per_axis(geom))
    _check(lib().gconv_step_ex(ctypes.byref(rec), int(dt), int(out_dt), x, w, bias or None, dy, y, dx, dw,
                               db or None, ws or None, int(ws_bytes), stream or None), "gconv_step_ex")


def gconv_bwd_weight_ex_ptr(geom, dt, x, dy, dw, db=0, ws=0, ws_bytes=0, stream=0):
    rec = geometry_record(geom)
    _check(lib().gconv_bwd_weight_ex(ctypes.byref(rec), int(dt), x, dy, dw, db or None, ws or None, int(ws_bytes),
                                     stream or None), "gconv_bwd_weight_ex")
