"""MI355X-native N-D transposed convolution (ONNX ConvTranspose).

This package is a thin Python binding over ``libconvtranspose.so``, whose C ABI is
declared in ``include/convtranspose.h``.  The binding only marshals arguments: it
resolves the output shape through the library, allocates Y with torch (torch supplies
device memory and the stream) and passes raw pointers.  Every step of the operator
runs in the library's HIP kernels; there is no CPU or PyTorch fallback, and a missing
library raises.

Operator: webgpu-kernels "ai.onnx.ConvTranspose" README (Description, Inputs,
Outputs, Attributes, Type constraints); channels-last input/output as on the ClikaRT
"conv_transpose" API page.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence, Tuple

import torch  # first: the library then binds to the HIP runtime torch has loaded

__all__ = [
    "ConvTransposeError", "ConvTransposePlan", "convtranspose_nd", "convtranspose_profile_events", "convtranspose_output_shape",
    "convtranspose_useful_macs", "convtranspose_select_kernel", "convtranspose_last_error",
    "convtranspose_kernel_name", "library_path", "load_library", "channels_last_empty",
    "to_channels_last", "KERNELS", "ACTIVATIONS", "convolution_nd", "convolution_output_shape",
    "IGEMM_TILES", "set_igemm_tile", "igemm_tile", "qlinear_convtranspose_nd", "PreparedCall",
    "NORM_ACTIVATIONS", "group_norm_nd", "group_norm_backward_nd", "dropout_nd", "embedding_nd",
    "embedding_backward_nd", "set_group_norm_control", "attention_nd", "attention_backward_nd", "rotary_nd", "adamw_nd",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
# CT_LIBRARY_PATH selects another build of the same library (e.g. one with host-side
# sanitizers); it must exist like the default one -- there is no fallback.
_LIB_PATH = os.environ.get("CT_LIBRARY_PATH") or os.path.join(_HERE, "libconvtranspose.so")
AUTO_PAD = {"NOTSET": 0, "SAME_UPPER": 1, "SAME_LOWER": 2, "VALID": 3}
KERNELS = {"auto": 0, "direct": 1, "grouped": 2, "igemm": 3, "none": 4}
# output activation fused into the kernels' output stage (ct_activation), with the number
# of parameters each takes: leaky_relu (slope,), clip (lower, upper)
ACTIVATIONS = {"identity": (0, 0), "relu": (1, 0), "leaky_relu": (2, 1), "clip": (3, 2)}
# group norm's activations: the same and SiLU
NORM_ACTIVATIONS = {**ACTIVATIONS, "silu": (4, 0)}
_DTYPES = {torch.float32: 0, torch.float16: 1}
# group norm, dropout, the embedding, attention, rotary positions and AdamW
_LAYER_DTYPES = {**_DTYPES, torch.bfloat16: 4}
_INDEX_DTYPES = {torch.int32: 5, torch.int64: 6}
_STATUS = {0: "CT_OK", 1: "CT_EINVAL", 2: "CT_ESHAPE", 3: "CT_EUNSUPPORTED", 4: "CT_EDEVICE"}
_lib = None


class ConvTransposeError(RuntimeError):
    """A library call returned a non-OK status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libconvtranspose.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(_LIB_PATH)
    i64p = ctypes.POINTER(ctypes.c_int64)
    vp = ctypes.c_void_p
    attrs = [ctypes.c_int, i64p, i64p, i64p, i64p, i64p, i64p, ctypes.c_int64]
    lib.convtranspose_output_shape.argtypes = [ctypes.c_int, i64p, i64p] + attrs + [i64p, i64p]
    lib.convtranspose_useful_macs.argtypes = [ctypes.c_int, i64p, i64p] + attrs + [
        ctypes.POINTER(ctypes.c_double)]
    call = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, i64p, vp, i64p, vp, vp, i64p] + attrs
    lib.convtranspose_nd.argtypes = call + [vp]
    lib.convtranspose_nd_with_kernel.argtypes = [ctypes.c_int] + call + [vp, ctypes.c_size_t, vp]
    lib.convtranspose_nd_fused.argtypes = [ctypes.c_int] + call + [ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                                                   vp, ctypes.c_size_t, vp]
    lib.convtranspose_nd_noalloc.argtypes = [ctypes.c_int] + call + [vp]
    lib.convtranspose_nd_noalloc.restype = ctypes.c_int
    lib.convtranspose_noalloc_max_workspace.argtypes = []
    lib.convtranspose_noalloc_max_workspace.restype = ctypes.c_size_t
    lib.convtranspose_workspace_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp,
                                                 i64p, i64p] + attrs + [ctypes.POINTER(ctypes.c_size_t)]
    lib.convtranspose_select_kernel.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, i64p,
                                                vp, i64p, vp, vp] + attrs
    for fn in ("convtranspose_output_shape", "convtranspose_useful_macs", "convtranspose_nd",
               "convtranspose_nd_with_kernel", "convtranspose_nd_fused", "convtranspose_select_kernel",
               "convtranspose_workspace_size"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.convtranspose_last_error.restype = ctypes.c_char_p
    lib.convtranspose_last_error.argtypes = []
    lib.convtranspose_kernel_name.restype = ctypes.c_char_p
    lib.convtranspose_kernel_name.argtypes = [ctypes.c_int]
    cattrs = [ctypes.c_int, i64p, i64p, i64p, i64p, ctypes.c_int64]  # forward convolution attributes
    lib.convolution_output_shape.argtypes = [ctypes.c_int, i64p, i64p] + cattrs + [i64p, i64p]
    lib.convolution_output_shape.restype = ctypes.c_int
    lib.convolution_nd.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, i64p, vp, i64p, vp,
                                   vp, i64p] + cattrs + [vp]
    lib.convolution_nd.restype = ctypes.c_int
    lib.convtranspose_profile_events.argtypes = [vp, vp]
    lib.convtranspose_profile_events.restype = ctypes.c_int
    c_i32, c_f32 = ctypes.c_int32, ctypes.c_float
    lib.qlinear_convtranspose_nd.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, ctypes.c_int, i64p, c_f32,
                                             c_i32, vp, ctypes.c_int, i64p, vp, vp, ctypes.c_int64, vp, vp,
                                             ctypes.c_int, i64p, c_f32, c_i32] + attrs + [vp]
    lib.qlinear_convtranspose_nd.restype = ctypes.c_int
    c_int, c_i64, c_u64, c_size = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    drop = [ctypes.c_double, c_u64, c_u64, vp]
    act = [c_int, c_f32, c_f32]
    lib.group_norm_nd.argtypes = [c_int, c_int, vp, i64p, c_i64, c_int, vp, vp, c_f32] + act + drop + [
        vp, vp, vp, vp, c_size, vp]
    lib.group_norm_backward_nd.argtypes = [c_int, c_int, vp, vp, i64p, c_i64, vp, vp, c_int, vp, vp] + act + drop + [
        vp, vp, vp, vp, c_size, vp]
    lib.group_norm_workspace_size.argtypes = [c_int, c_int, i64p, c_i64, c_int, ctypes.POINTER(c_size)]
    lib.group_norm_set_control.argtypes = [c_int, c_int]
    lib.group_norm_set_control.restype = c_int
    lib.dropout_nd.argtypes = [c_int, c_i64, vp, vp, vp] + drop + [vp]
    lib.embedding_nd.argtypes = [c_int, c_int, c_i64, vp, c_i64, c_i64, vp, c_f32, vp, vp]
    lib.embedding_backward_nd.argtypes = [c_int, c_int, c_i64, vp, c_i64, c_i64, vp, c_f32, c_i64, c_int, vp, vp, c_size,
                                          vp]
    lib.embedding_workspace_size.argtypes = [c_i64, c_i64, c_i64, ctypes.POINTER(c_size)]
    c_f64 = ctypes.c_double
    mask = [c_f32, c_int, vp, vp]  # scale, causal, lengths, starts
    lib.attention_nd.argtypes = [c_int, i64p, c_i64, c_i64] + [vp, i64p] * 3 + mask + [vp, vp, vp, c_size, vp]
    lib.attention_backward_nd.argtypes = [c_int, i64p, c_i64, c_i64] + [vp, i64p] * 5 + [vp] + mask + [
        vp, vp, vp, vp, c_size, vp]
    lib.attention_workspace_size.argtypes = [c_int, i64p, c_i64, c_i64, c_int, ctypes.POINTER(c_size)]
    lib.rotary_nd.argtypes = [c_int, i64p, vp, i64p, c_int, c_int, vp, i64p, i64p, c_f64, c_int, c_int, c_int, vp, i64p, vp]
    lib.adamw_nd.argtypes = [c_int, c_int, c_int, c_int, c_i64, vp, c_f64, vp, c_f64, c_f64, c_f64, c_i64, vp, c_f64, vp, vp]
    for fn in ("group_norm_nd", "group_norm_backward_nd", "group_norm_workspace_size", "dropout_nd", "embedding_nd",
               "embedding_backward_nd", "embedding_workspace_size", "attention_nd", "attention_backward_nd",
               "attention_workspace_size", "rotary_nd", "adamw_nd"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.convtranspose_set_igemm_tile.argtypes = [ctypes.c_int]
    lib.convtranspose_set_igemm_tile.restype = ctypes.c_int
    lib.convtranspose_igemm_tile.argtypes = []
    lib.convtranspose_igemm_tile.restype = ctypes.c_int
    _lib = lib
    return lib


def convtranspose_last_error() -> str:
    return load_library().convtranspose_last_error().decode(errors="replace")


def convtranspose_kernel_name(kernel: int) -> str:
    return load_library().convtranspose_kernel_name(int(kernel)).decode()


def _i64(v: Optional[Sequence[int]]):
    if v is None:
        return None
    v = [int(t) for t in v]
    return (ctypes.c_int64 * max(1, len(v)))(*v)


def _attr_args(nsp, auto_pad="NOTSET", strides=None, dilations=None, pads=None, output_padding=None,
               output_shape=None, kernel_shape=None, group=1):
    lens = dict(strides=nsp, dilations=nsp, pads=2 * nsp, output_padding=nsp, output_shape=nsp,
                kernel_shape=nsp)
    vals = dict(strides=strides, dilations=dilations, pads=pads, output_padding=output_padding,
                output_shape=output_shape, kernel_shape=kernel_shape)
    for k, v in vals.items():
        if v is not None and len(v) != lens[k]:
            raise ConvTransposeError(1, f"{k} must have {lens[k]} entries")
    if auto_pad not in AUTO_PAD:
        raise ConvTransposeError(1, f"unknown auto_pad {auto_pad!r}")
    return [AUTO_PAD[auto_pad]] + [_i64(vals[k]) for k in
                                   ("strides", "dilations", "pads", "output_padding", "output_shape",
                                    "kernel_shape")] + [int(group)]


def _raise(st: int):
    raise ConvTransposeError(st, convtranspose_last_error())


def convtranspose_output_shape(x_shape, w_shape, **attrs) -> Tuple[Tuple[int, ...], Tuple[int, ...]]:
    """Resolved Y shape (N, M, O1..On) and applied pads (begins, then ends)."""
    lib = load_library()
    nsp = len(x_shape) - 2
    if len(w_shape) != len(x_shape):
        raise ConvTransposeError(1, "W must have the same rank as X")
    ys = (ctypes.c_int64 * (nsp + 2))()
    pd = (ctypes.c_int64 * max(1, 2 * nsp))()
    st = lib.convtranspose_output_shape(nsp, _i64(x_shape), _i64(w_shape), *_attr_args(nsp, **attrs),
                                        ys, pd)
    if st:
        _raise(st)
    return tuple(ys), tuple(pd[: 2 * nsp])


def convtranspose_useful_macs(x_shape, w_shape, **attrs) -> int:
    """Useful MACs: in-range (input sample, tap) pairs times N * C/group * M."""
    lib = load_library()
    nsp = len(x_shape) - 2
    out = ctypes.c_double(0.0)
    st = lib.convtranspose_useful_macs(nsp, _i64(x_shape), _i64(w_shape), *_attr_args(nsp, **attrs),
                                       ctypes.byref(out))
    if st:
        _raise(st)
    return int(out.value)


def _expected_cl_strides(shape):
    """Strides of a dense channels-last tensor with logical shape (N, C, D1..Dn)."""
    N, C, sp = shape[0], shape[1], list(shape[2:])
    st = [0] * len(shape)
    st[1] = 1
    acc = C
    for a in range(len(sp) - 1, -1, -1):
        st[2 + a] = acc
        acc *= sp[a]
    st[0] = acc
    return st


def _dense(t: torch.Tensor, channels_last: bool) -> bool:
    if t.numel() == 0:
        return True  # nothing is read or written
    if not channels_last:
        return t.is_contiguous()
    want = _expected_cl_strides(t.shape)
    return all(sz <= 1 or s == w for sz, s, w in zip(t.shape, t.stride(), want))


def channels_last_empty(shape, dtype, device) -> torch.Tensor:
    """Uninitialised tensor of logical shape (N, C, D..) stored (N, D.., C)."""
    nsp = len(shape) - 2
    phys = torch.empty((shape[0],) + tuple(shape[2:]) + (shape[1],), dtype=dtype, device=device)
    return phys.permute(0, nsp + 1, *range(1, nsp + 1))


def to_channels_last(t: torch.Tensor) -> torch.Tensor:
    """Dense channels-last copy of a logical (N, C, D..) tensor."""
    nsp = t.dim() - 2
    return t.permute(0, *range(2, nsp + 2), 1).contiguous().permute(0, nsp + 1, *range(1, nsp + 1))


def _check_tensor(name, t, device, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ConvTransposeError(1, f"{name} must be on a HIP device (got {t.device})")
    if t.device != device:
        raise ConvTransposeError(1, f"{name} is on {t.device}, x is on {device}")
    if t.dtype != dtype:
        raise ConvTransposeError(3, f"{name} has dtype {t.dtype}, x has {dtype}")


def _call_args(x, w, bias, y, attrs):
    nsp = x.dim() - 2
    ptr = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    return nsp, ptr(x), _i64(x.shape), ptr(w), _i64(w.shape), ptr(bias), ptr(y), _attr_args(nsp, **attrs)


def convtranspose_select_kernel(x, w, bias=None, *, channels_last=False, **attrs) -> str:
    """Name of the kernel family the dispatcher would run for these tensors."""
    lib = load_library()
    if x.dtype not in _DTYPES:
        raise ConvTransposeError(3, f"dtype {x.dtype} is not served")
    nsp, xp, xs, wp, ws, bp, _, at = _call_args(x, w, bias, None, attrs)
    yshape, _ = convtranspose_output_shape(tuple(x.shape), tuple(w.shape), **attrs)
    # alignment of y is that of a fresh torch allocation (256 B)
    k = lib.convtranspose_select_kernel(_DTYPES[x.dtype], nsp, int(channels_last), xp, xs, wp, ws, bp,
                                        ctypes.c_void_p(256), *at)
    if k < 0:
        raise ConvTransposeError(1, convtranspose_last_error())
    return convtranspose_kernel_name(k)


class ConvTransposePlan:
    """One ConvTranspose with its arguments resolved and marshalled once.

    Construction validates the tensors, resolves Y's shape, allocates Y (unless ``out``
    is given) and the implicit-GEMM scratch, and builds the C argument list; each call
    then enqueues the operation on ``stream`` (default: torch's current stream of x's
    device at construction) with a single C call.  Repeated calls reuse Y and the
    scratch, so they must be ordered on one stream.
    """

    def __init__(self, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                 auto_pad: str = "NOTSET", strides=None, dilations=None, pads=None,
                 output_padding=None, output_shape=None, kernel_shape=None, group: int = 1,
                 channels_last: bool = False, out: Optional[torch.Tensor] = None,
                 kernel: str = "auto", stream: Optional[torch.cuda.Stream] = None,
                 activation: str = "identity", act_params: Sequence[float] = ()):
        lib = load_library()
        if activation not in ACTIVATIONS:
            raise ConvTransposeError(1, f"unknown activation {activation!r}")
        act_kind, act_n = ACTIVATIONS[activation]
        if len(act_params) != act_n:
            raise ConvTransposeError(1, f"{activation} takes {act_n} parameter(s)")
        act_p = [float(v) for v in act_params] + [0.0] * (2 - act_n)
        if x.dtype not in _DTYPES:
            raise ConvTransposeError(3, f"dtype {x.dtype} is not served (float32, float16)")
        if x.dim() < 3 or x.dim() > 5:
            raise ConvTransposeError(1, "x must have rank 3, 4 or 5")
        dev = x.device
        _check_tensor("x", x, dev, x.dtype)
        _check_tensor("w", w, dev, x.dtype)
        if w.dim() != x.dim():
            raise ConvTransposeError(1, "W must have the same rank as X")
        if bias is not None:
            _check_tensor("bias", bias, dev, x.dtype)
            if bias.dim() != 1 or not bias.is_contiguous():
                raise ConvTransposeError(1, "bias must be a dense 1-D tensor")
            if bias.shape[0] != w.shape[1] * int(group):
                raise ConvTransposeError(1, "bias length must equal M = W.shape[1] * group")
        if not _dense(x, channels_last):
            raise ConvTransposeError(1, "x is not dense in the requested layout")
        if not w.is_contiguous():
            raise ConvTransposeError(1, "w must be contiguous")
        if kernel not in KERNELS:
            raise ConvTransposeError(1, f"unknown kernel {kernel!r}")
        attrs = dict(auto_pad=auto_pad, strides=strides, dilations=dilations, pads=pads,
                     output_padding=output_padding, output_shape=output_shape,
                     kernel_shape=kernel_shape, group=group)
        yshape, _ = convtranspose_output_shape(tuple(x.shape), tuple(w.shape), **attrs)
        if out is None:
            out = (channels_last_empty(yshape, x.dtype, dev) if channels_last
                   else torch.empty(yshape, dtype=x.dtype, device=dev))
        else:
            _check_tensor("out", out, dev, x.dtype)
            if tuple(out.shape) != tuple(yshape):
                raise ConvTransposeError(2, f"out has shape {tuple(out.shape)}, expected {yshape}")
            if not _dense(out, channels_last):
                raise ConvTransposeError(1, "out is not dense in the requested layout")
        nsp, xp, xs, wp, ws, bp, yp, at = _call_args(x, w, bias, out, attrs)
        nbytes = ctypes.c_size_t(0)
        st = lib.convtranspose_workspace_size(KERNELS[kernel], _DTYPES[x.dtype], nsp, int(channels_last), xp,
                                              xs, ws, *at, ctypes.byref(nbytes))
        if st:
            _raise(st)
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        self.scratch = None
        if nbytes.value:
            with torch.cuda.stream(self.stream):
                self.scratch = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
        self.out = out
        self.device = dev
        self._keep = (x, w, bias)  # the pointers below stay valid while the plan lives
        self._fn = lib.convtranspose_nd_fused
        self._args = (KERNELS[kernel], _DTYPES[x.dtype], nsp, int(channels_last), xp, xs, wp, ws, bp, yp,
                      _i64(yshape), *at, act_kind, act_p[0], act_p[1],
                      ctypes.c_void_p(self.scratch.data_ptr()) if self.scratch is not None else None,
                      nbytes.value, ctypes.c_void_p(self.stream.cuda_stream))

    def __call__(self) -> torch.Tensor:
        with torch.cuda.device(self.device):
            st = self._fn(*self._args)
        if st:
            _raise(st)
        return self.out


def convtranspose_nd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                     auto_pad: str = "NOTSET", strides=None, dilations=None, pads=None,
                     output_padding=None, output_shape=None, kernel_shape=None, group: int = 1,
                     channels_last: bool = False, out: Optional[torch.Tensor] = None,
                     kernel: str = "auto", stream: Optional[torch.cuda.Stream] = None,
                     activation: str = "identity", act_params: Sequence[float] = ()) -> torch.Tensor:
    """Y = ConvTranspose(X, W, bias) on the GPU, enqueued on ``stream`` (default: torch's
    current stream of x's device).

    x: logical (N, C, D1..Dn) float32/float16 on a HIP device; dense NC.. storage, or
    dense N..C storage when ``channels_last`` (see ``to_channels_last``).
    w: (C, M/group, k1..kn) dense.  bias: (M,) or None.  Y is allocated (or ``out`` is
    used) with the same layout convention as x.  ``kernel`` forces a kernel family.
    ``activation`` ("identity", "relu", "leaky_relu" with ``act_params=(slope,)``, "clip"
    with ``act_params=(lower, upper)``) is applied to every output in float32, after the
    bias and before the one rounding, inside the kernel that computes it.
    """
    return ConvTransposePlan(x, w, bias, auto_pad=auto_pad, strides=strides, dilations=dilations,
                             pads=pads, output_padding=output_padding, output_shape=output_shape,
                             kernel_shape=kernel_shape, group=group, channels_last=channels_last,
                             out=out, kernel=kernel, stream=stream, activation=activation,
                             act_params=act_params)()


def convtranspose_nd_noalloc(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                             out: torch.Tensor, auto_pad: str = "NOTSET", strides=None, dilations=None, pads=None,
                             output_padding=None, output_shape=None, kernel_shape=None, group: int = 1,
                             channels_last: bool = False, kernel: str = "auto",
                             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The C entry point ``convtranspose_nd_noalloc``: Y = ConvTranspose(X, W, bias) into the
    caller's ``out`` with the library's fixed device workspace, so nothing is allocated
    (neither here nor in the library).  Arguments as for ``convtranspose_nd``; ``out`` is
    required.  Calls on one device share the workspace: order them on one stream."""
    lib = load_library()
    if x.dtype not in _DTYPES:
        raise ConvTransposeError(3, f"dtype {x.dtype} is not served (float32, float16)")
    if kernel not in KERNELS:
        raise ConvTransposeError(1, f"unknown kernel {kernel!r}")
    dev = x.device
    for name, t in (("x", x), ("w", w), ("out", out)) + ((("bias", bias),) if bias is not None else ()):
        _check_tensor(name, t, dev, x.dtype)
    if not _dense(x, channels_last) or not _dense(out, channels_last) or not w.is_contiguous():
        raise ConvTransposeError(1, "x, out and w must be dense in the requested layout")
    attrs = dict(auto_pad=auto_pad, strides=strides, dilations=dilations, pads=pads,
                 output_padding=output_padding, output_shape=output_shape,
                 kernel_shape=kernel_shape, group=group)
    nsp, xp, xs, wp, ws, bp, yp, at = _call_args(x, w, bias, out, attrs)
    st_ = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        st = lib.convtranspose_nd_noalloc(KERNELS[kernel], _DTYPES[x.dtype], nsp, int(channels_last), xp, xs, wp, ws,
                                          bp, yp, _i64(tuple(out.shape)), *at, ctypes.c_void_p(st_.cuda_stream))
    if st:
        _raise(st)
    return out


IGEMM_TILES = ("256x256", "128x256", "64x512", "64x256", "64x128", "allphase", "tapsplit")


def set_igemm_tile(tile: Optional[str]) -> None:
    """Force one block shape of the float16 MFMA kernel (a name from IGEMM_TILES, output
    channels x output pixels), or None for the automatic choice.  Process-wide."""
    lib = load_library()
    st = lib.convtranspose_set_igemm_tile(-1 if tile is None else IGEMM_TILES.index(tile))
    if st:
        _raise(st)


def igemm_tile() -> Optional[str]:
    """The forced block shape of the float16 MFMA kernel, or None (automatic)."""
    t = load_library().convtranspose_igemm_tile()
    return None if t < 0 else IGEMM_TILES[t]


def convtranspose_profile_events(before: Optional[torch.cuda.Event], after: Optional[torch.cuda.Event]):
    """Have later calls on this thread record ``before``/``after`` around their dominant
    kernel (timing events created with ``enable_timing=True``); None, None turns it off."""
    lib = load_library()
    handles = []
    for ev in (before, after):
        if ev is None:
            handles.append(None)
            continue
        if not ev.cuda_event:
            ev.record()  # torch creates the HIP event on first record
        handles.append(ctypes.c_void_p(ev.cuda_event))
    st = lib.convtranspose_profile_events(*handles)
    if st:
        _raise(st)


# ------------------------------------------------------------------------------------
# The forward convolution with the same W (the adjoint of the transposed convolution)
# ------------------------------------------------------------------------------------
def _conv_attr_args(nsp, auto_pad="NOTSET", strides=None, dilations=None, pads=None, kernel_shape=None, group=1):
    lens = dict(strides=nsp, dilations=nsp, pads=2 * nsp, kernel_shape=nsp)
    vals = dict(strides=strides, dilations=dilations, pads=pads, kernel_shape=kernel_shape)
    for k, v in vals.items():
        if v is not None and len(v) != lens[k]:
            raise ConvTransposeError(1, f"{k} must have {lens[k]} entries")
    if auto_pad not in AUTO_PAD:
        raise ConvTransposeError(1, f"unknown auto_pad {auto_pad!r}")
    return [AUTO_PAD[auto_pad], _i64(strides), _i64(dilations), _i64(pads), _i64(kernel_shape), int(group)]


def convolution_output_shape(x_shape, w_shape, **attrs) -> Tuple[Tuple[int, ...], Tuple[int, ...]]:
    """Forward convolution: resolved Y shape (N, M, O1..On) and applied pads."""
    lib = load_library()
    nsp = len(x_shape) - 2
    if len(w_shape) != len(x_shape):
        raise ConvTransposeError(1, "W must have the same rank as X")
    ys = (ctypes.c_int64 * (nsp + 2))()
    pd = (ctypes.c_int64 * max(1, 2 * nsp))()
    st = lib.convolution_output_shape(nsp, _i64(x_shape), _i64(w_shape), *_conv_attr_args(nsp, **attrs), ys, pd)
    if st:
        _raise(st)
    return tuple(ys), tuple(pd[: 2 * nsp])


def convolution_nd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                   auto_pad: str = "NOTSET", strides=None, dilations=None, pads=None, kernel_shape=None,
                   group: int = 1, channels_last: bool = False, out: Optional[torch.Tensor] = None,
                   kernel: str = "auto", stream: Optional[torch.cuda.Stream] = None,
                   _prepare_only: bool = False) -> torch.Tensor:
    """Y = Conv(X, W, bias) on the GPU (ONNX Conv; W is (M, C/group, k1..kn)), the adjoint of
    ``convtranspose_nd`` with the same W.  ``kernel``: "auto", "direct" or "igemm" (the
    MFMA path: stride 1, or strided with dilation 1 through the input phases)."""
    lib = load_library()
    if x.dtype not in _DTYPES:
        raise ConvTransposeError(3, f"dtype {x.dtype} is not served (float32, float16)")
    if x.dim() < 3 or x.dim() > 5 or w.dim() != x.dim():
        raise ConvTransposeError(1, "x and w must have the same rank, 3 to 5")
    dev = x.device
    _check_tensor("x", x, dev, x.dtype)
    _check_tensor("w", w, dev, x.dtype)
    if bias is not None:
        _check_tensor("bias", bias, dev, x.dtype)
        if bias.dim() != 1 or not bias.is_contiguous() or bias.shape[0] != w.shape[0]:
            raise ConvTransposeError(1, "bias must be a dense 1-D tensor of length M = W.shape[0]")
    if not _dense(x, channels_last) or not w.is_contiguous():
        raise ConvTransposeError(1, "x (in the requested layout) and w must be dense")
    if kernel not in ("auto", "direct", "igemm"):
        raise ConvTransposeError(1, f"unknown kernel {kernel!r}")
    attrs = dict(auto_pad=auto_pad, strides=strides, dilations=dilations, pads=pads, kernel_shape=kernel_shape,
                 group=group)
    yshape, _ = convolution_output_shape(tuple(x.shape), tuple(w.shape), **attrs)
    if out is None:
        out = (channels_last_empty(yshape, x.dtype, dev) if channels_last
               else torch.empty(yshape, dtype=x.dtype, device=dev))
    else:
        _check_tensor("out", out, dev, x.dtype)
        if tuple(out.shape) != tuple(yshape) or not _dense(out, channels_last):
            raise ConvTransposeError(2, f"out must be dense with shape {yshape}")
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    nsp = x.dim() - 2
    ptr = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    args = (KERNELS[kernel], _DTYPES[x.dtype], nsp, int(channels_last), ptr(x), _i64(x.shape), ptr(w), _i64(w.shape),
            ptr(bias), ptr(out), _i64(yshape), *_conv_attr_args(nsp, **attrs), ctypes.c_void_p(stream.cuda_stream))
    if _prepare_only:
        return lib.convolution_nd, args, out
    with torch.cuda.device(dev):
        st = lib.convolution_nd(*args)
    if st:
        _raise(st)
    return out


_QTYPES = {torch.int8: 2, torch.uint8: 3}


def qlinear_convtranspose_nd(x: torch.Tensor, x_scale: float, x_zero_point: int, w: torch.Tensor,
                             w_scale: torch.Tensor, w_zero_point: torch.Tensor, y_scale: float, y_zero_point: int,
                             y_dtype: torch.dtype = torch.uint8, bias: Optional[torch.Tensor] = None, *,
                             auto_pad: str = "NOTSET", strides=None, dilations=None, pads=None, output_padding=None,
                             output_shape=None, kernel_shape=None, group: int = 1, channels_last: bool = False,
                             out: Optional[torch.Tensor] = None, kernel: str = "auto",
                             stream: Optional[torch.cuda.Stream] = None, _prepare_only: bool = False) -> torch.Tensor:
    """Quantized ConvTranspose (QLinear scheme) on the GPU: uint8/int8 x, w and y; x and y
    quantized per tensor (host scalars), w per tensor or per output channel (w_scale
    float32 and w_zero_point of w's dtype, 1 or M values, on x's device); bias int32."""
    lib = load_library()
    for name, t in (("x", x), ("w", w), ("w_zero_point", w_zero_point)):
        if t.dtype not in _QTYPES:
            raise ConvTransposeError(3, f"{name} must be uint8 or int8 (got {t.dtype})")
    if y_dtype not in _QTYPES:
        raise ConvTransposeError(3, f"y_dtype must be uint8 or int8 (got {y_dtype})")
    if w_zero_point.dtype != w.dtype:
        raise ConvTransposeError(3, "w_zero_point must have w's dtype")
    if x.dim() < 3 or x.dim() > 5 or w.dim() != x.dim():
        raise ConvTransposeError(1, "x and w must have the same rank, 3 to 5")
    dev = x.device
    _check_tensor("x", x, dev, x.dtype)
    _check_tensor("w", w, dev, w.dtype)
    _check_tensor("w_scale", w_scale, dev, torch.float32)
    _check_tensor("w_zero_point", w_zero_point, dev, w.dtype)
    if w_scale.dim() != 1 or w_zero_point.dim() != 1 or w_scale.numel() != w_zero_point.numel() \
            or not w_scale.is_contiguous() or not w_zero_point.is_contiguous():
        raise ConvTransposeError(1, "w_scale and w_zero_point must be dense 1-D tensors of the same length")
    if bias is not None:
        _check_tensor("bias", bias, dev, torch.int32)
        if bias.dim() != 1 or not bias.is_contiguous():
            raise ConvTransposeError(1, "bias must be a dense 1-D int32 tensor")
    if not _dense(x, channels_last) or not w.is_contiguous():
        raise ConvTransposeError(1, "x (in the requested layout) and w must be dense")
    if kernel not in KERNELS:
        raise ConvTransposeError(1, f"unknown kernel {kernel!r}")
    attrs = dict(auto_pad=auto_pad, strides=strides, dilations=dilations, pads=pads, output_padding=output_padding,
                 output_shape=output_shape, kernel_shape=kernel_shape, group=group)
    yshape, _ = convtranspose_output_shape(tuple(x.shape), tuple(w.shape), **attrs)
    if out is None:
        out = (channels_last_empty(yshape, y_dtype, dev) if channels_last
               else torch.empty(yshape, dtype=y_dtype, device=dev))
    else:
        _check_tensor("out", out, dev, y_dtype)
        if tuple(out.shape) != tuple(yshape) or not _dense(out, channels_last):
            raise ConvTransposeError(2, f"out must be dense with shape {yshape}")
    stream = stream if stream is not None else torch.cuda.current_stream(dev)
    nsp = x.dim() - 2
    ptr = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    args = (KERNELS[kernel], nsp, int(channels_last), ptr(x), _QTYPES[x.dtype], _i64(x.shape), float(x_scale),
            int(x_zero_point), ptr(w), _QTYPES[w.dtype], _i64(w.shape), ptr(w_scale), ptr(w_zero_point),
            w_scale.numel(), ptr(bias), ptr(out), _QTYPES[y_dtype], _i64(yshape), float(y_scale), int(y_zero_point),
            *_attr_args(nsp, **attrs), ctypes.c_void_p(stream.cuda_stream))
    if _prepare_only:
        return lib.qlinear_convtranspose_nd, args, out
    with torch.cuda.device(dev):
        st = lib.qlinear_convtranspose_nd(*args)
    if st:
        _raise(st)
    return out


# ------------------------------------------------------------------------------------
# The other operators of a decoder layer: group norm with an activation, dropout, embedding
# ------------------------------------------------------------------------------------
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _call(fn, args, out, keep, prepare_only):
    """Run a marshalled C call, or hand it to PreparedCall with what it keeps alive."""
    if prepare_only:
        return fn, args, out, keep
    first = out[0] if isinstance(out, tuple) else out
    with torch.cuda.device(first.device):
        st = fn(*args)
    if st:
        _raise(st)
    return out


def _scratch(nbytes: int, device, prepare_only):
    """A prepared call's own workspace; a direct call takes the library's pool."""
    if not prepare_only or not nbytes:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _on(stream):
    """Memory of new outputs comes from the stream that writes them: torch may hand out what
    the current stream still uses."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _stream_ptr(stream, device):
    return ctypes.c_void_p((stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream)


def _dropout_args(p, seed, offset, step, device):
    if not 0.0 <= float(p) <= 1.0:
        raise ConvTransposeError(1, "the dropout probability must lie in [0, 1]")
    for name, v in (("seed", seed), ("offset", offset)):
        if not 0 <= int(v) < 1 << 64:
            raise ConvTransposeError(1, f"{name} must be an unsigned 64-bit number")
    if step is not None:
        _check_tensor("step", step, device, torch.int64)
        if step.numel() != 1:
            raise ConvTransposeError(1, "step must hold one int64")
    return [float(p), int(seed), int(offset), _ptr(step)]


def _norm_args(x, groups, gamma, beta, activation, act_params):
    """Checks both directions of group norm share; (type code of the parameters, act arguments)."""
    if x.dtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, f"dtype {x.dtype} is not served (float32, float16, bfloat16)")
    if x.dim() < 3 or x.dim() > 5:
        raise ConvTransposeError(1, "x must have rank 3, 4 or 5")
    _check_tensor("x", x, x.device, x.dtype)
    if not _dense(x, True):
        raise ConvTransposeError(1, "x is not dense channels-last")
    if int(groups) < 1 or x.shape[1] % int(groups):
        raise ConvTransposeError(1, "groups must be at least 1 and divide the channels")
    if activation not in NORM_ACTIVATIONS:
        raise ConvTransposeError(1, f"unknown activation {activation!r}")
    kind, n = NORM_ACTIVATIONS[activation]
    if len(act_params) != n:
        raise ConvTransposeError(1, f"{activation} takes {n} parameter(s)")
    ptype = next((t.dtype for t in (gamma, beta) if t is not None), torch.float32)
    if ptype not in (x.dtype, torch.float32):
        raise ConvTransposeError(3, f"gamma and beta must be float32 or {x.dtype} (got {ptype})")
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None:
            _check_tensor(name, t, x.device, ptype)
            if t.dim() != 1 or not t.is_contiguous() or t.shape[0] != x.shape[1]:
                raise ConvTransposeError(1, f"{name} must be a dense 1-D tensor with one value a channel")
    return _LAYER_DTYPES[ptype], [kind] + [float(v) for v in act_params] + [0.0] * (2 - n)


def _norm_workspace(x, groups, backward):
    nbytes = ctypes.c_size_t(0)
    st = load_library().group_norm_workspace_size(_LAYER_DTYPES[x.dtype], x.dim() - 2, _i64(x.shape), int(groups),
                                                  int(backward), ctypes.byref(nbytes))
    if st:
        _raise(st)
    return nbytes.value


def _channels_last_like(name, t, x):
    """A caller's output (None: a new one) with x's shape, type and channels-last storage."""
    if t is None:
        return channels_last_empty(tuple(x.shape), x.dtype, x.device)
    _check_tensor(name, t, x.device, x.dtype)
    if t.shape != x.shape:
        raise ConvTransposeError(2, f"{name} has shape {tuple(t.shape)}, expected {tuple(x.shape)}")
    if not _dense(t, True):
        raise ConvTransposeError(1, f"{name} is not dense channels-last")
    return t


def group_norm_nd(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None,
                  beta: Optional[torch.Tensor] = None, *, eps: float = 1e-5, activation: str = "identity",
                  act_params: Sequence[float] = (), dropout_p: float = 0.0, seed: int = 0, offset: int = 0,
                  step: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None,
                  _prepare_only: bool = False) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): group norm over ``groups`` channel groups, an activation and dropout, in
    one call, channels-last.

    x: logical (N, C, D1..Dn) float32/float16/bfloat16, dense N, D.., C storage.  gamma, beta:
    (C,) in x's type or float32, or None.  ``activation``: a name from NORM_ACTIVATIONS.
    ``dropout_p``, ``seed``, ``offset``, ``step``: dropout of the activation's output as by
    ``dropout_nd`` (elements in storage order).  y has x's layout (``out``: the caller's, may
    be x); mean and rstd are (N, groups) float32, for ``group_norm_backward_nd``."""
    lib = load_library()
    ptype, act = _norm_args(x, groups, gamma, beta, activation, act_params)
    drop = _dropout_args(dropout_p, seed, offset, step, x.device)
    nbytes = _norm_workspace(x, groups, False) if _prepare_only else 0
    with _on(stream):
        out = _channels_last_like("out", out, x)
        new = torch.empty if x.numel() else torch.zeros
        mean, rstd = new((2, x.shape[0], int(groups)), dtype=torch.float32, device=x.device).unbind(0)
        ws, wsb = _scratch(nbytes, x.device, _prepare_only)
    args = (_LAYER_DTYPES[x.dtype], x.dim() - 2, _ptr(x), _i64(x.shape), int(groups), ptype, _ptr(gamma), _ptr(beta),
            float(eps), *act, *drop, _ptr(out), _ptr(mean), _ptr(rstd), _ptr(ws), wsb, _stream_ptr(stream, x.device))
    return _call(lib.group_norm_nd, args, (out, mean, rstd), ws, _prepare_only)


def group_norm_backward_nd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, groups: int,
                           gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None, *,
                           activation: str = "identity", act_params: Sequence[float] = (), dropout_p: float = 0.0,
                           seed: int = 0, offset: int = 0, step: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                           _prepare_only: bool = False
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dgamma, dbeta): the gradient of ``group_norm_nd`` from y's gradient dy, its input x
    and the statistics it returned, with the same parameters, activation and dropout.
    dgamma and dbeta have gamma's and beta's type and are None where those are.  ``out``:
    the caller's dx (may be dy or x)."""
    lib = load_library()
    ptype, act = _norm_args(x, groups, gamma, beta, activation, act_params)
    drop = _dropout_args(dropout_p, seed, offset, step, x.device)
    _channels_last_like("dy", dy, x)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _check_tensor(name, t, x.device, torch.float32)
        if tuple(t.shape) != (x.shape[0], int(groups)) or not t.is_contiguous():
            raise ConvTransposeError(1, f"{name} must be a dense (N, groups) tensor")
    nbytes = _norm_workspace(x, groups, True) if _prepare_only else 0
    with _on(stream):
        out = _channels_last_like("out", out, x)
        dgamma, dbeta = (None if t is None else torch.empty_like(t) for t in (gamma, beta))
        ws, wsb = _scratch(nbytes, x.device, _prepare_only)
    args = (_LAYER_DTYPES[x.dtype], x.dim() - 2, _ptr(dy), _ptr(x), _i64(x.shape), int(groups), _ptr(mean), _ptr(rstd),
            ptype, _ptr(gamma), _ptr(beta), *act, *drop, _ptr(out), _ptr(dgamma), _ptr(dbeta), _ptr(ws), wsb,
            _stream_ptr(stream, x.device))
    return _call(lib.group_norm_backward_nd, args, (out, dgamma, dbeta), ws, _prepare_only)


def set_group_norm_control(one_block: bool = True, join: Optional[bool] = None) -> None:
    """Group norm's kernels, for tests and tuning (process-wide): ``one_block`` False takes two
    passes even where a group fits one block; ``join`` True or False joins the first pass's
    partial sums in a kernel of its own or in the second pass (None: by their number)."""
    st = load_library().group_norm_set_control(-1 if one_block else 0, -1 if join is None else int(join))
    if st:
        _raise(st)


def _storage_order(t: torch.Tensor):
    """Strides of the axes longer than one when t fills its storage without gaps or overlap,
    else None."""
    if t.numel() == 0:
        return ()
    axes = sorted((st, sz) for sz, st in zip(t.shape, t.stride()) if sz > 1)
    acc = 1
    for st, sz in axes:
        if st != acc:
            return None
        acc *= sz
    return tuple(st for sz, st in zip(t.shape, t.stride()) if sz > 1)


def dropout_nd(x: torch.Tensor, p: float, *, seed: int, offset: int = 0, step: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None, _prepare_only: bool = False) -> torch.Tensor:
    """y = (residual +) dropout(x): elements drop with probability p (in steps of 2^-16), the
    others are scaled to keep the expectation.  The mask is a function of (seed, offset,
    place in storage) and is never stored: the gradient of x is
    ``dropout_nd(dy, p, seed=seed, offset=offset)``, that of the residual dy itself.

    x: float32/float16/bfloat16 of any rank, dense in some order of its axes; residual and
    out have x's strides (out may be x or residual).  Calls that shall be independent take
    different offsets (or seeds).  ``step``: one int64 on the device that is added to the
    offset when the kernel runs, so a captured or prepared call can draw anew each time."""
    lib = load_library()
    if x.dtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, f"dtype {x.dtype} is not served (float32, float16, bfloat16)")
    _check_tensor("x", x, x.device, x.dtype)
    drop = _dropout_args(p, seed, offset, step, x.device)
    order = _storage_order(x)
    if order is None:
        raise ConvTransposeError(1, "x must be dense")
    if out is None:
        with _on(stream):
            out = torch.empty_like(x)  # keeps a dense tensor's strides
    for name, t in (("residual", residual), ("out", out)):
        if t is not None:
            _check_tensor(name, t, x.device, x.dtype)
            if t.shape != x.shape:
                raise ConvTransposeError(2, f"{name} has shape {tuple(t.shape)}, expected {tuple(x.shape)}")
            if _storage_order(t) != order:
                raise ConvTransposeError(1, f"{name} must have x's strides")
    args = (_LAYER_DTYPES[x.dtype], x.numel(), _ptr(x), _ptr(residual), _ptr(out), *drop, _stream_ptr(stream, x.device))
    return _call(lib.dropout_nd, args, out, None, _prepare_only)


def _check_ids(ids, device):
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in _INDEX_DTYPES:
        raise ConvTransposeError(3, f"ids must be int32 or int64 (got {ids.dtype})")
    _check_tensor("ids", ids, device, ids.dtype)
    if not ids.is_contiguous():
        raise ConvTransposeError(1, "ids must be contiguous")


def embedding_nd(ids: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None, _prepare_only: bool = False) -> torch.Tensor:
    """y = scale * table[ids], of shape ids.shape + (width,).  ids: int32/int64 of any rank,
    contiguous; table: (rows, width) float32/float16/bfloat16, contiguous.  An id outside
    [0, rows) gives zeros.  For an (N, D1..Dn) grid of ids, ``y.movedim(-1, 1)`` is the
    channels-last (N, width, D1..Dn) tensor the convolutions take."""
    lib = load_library()
    if table.dtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, f"dtype {table.dtype} is not served (float32, float16, bfloat16)")
    _check_tensor("table", table, table.device, table.dtype)
    if table.dim() != 2 or not table.is_contiguous():
        raise ConvTransposeError(1, "table must be a dense (rows, width) tensor")
    _check_ids(ids, table.device)
    shape = tuple(ids.shape) + (table.shape[1],)
    if out is None:
        with _on(stream):
            out = torch.empty(shape, dtype=table.dtype, device=table.device)
    else:
        _check_tensor("out", out, table.device, table.dtype)
        if tuple(out.shape) != shape or not out.is_contiguous():
            raise ConvTransposeError(2, f"out must be dense with shape {shape}")
    args = (_LAYER_DTYPES[table.dtype], _INDEX_DTYPES[ids.dtype], ids.numel(), _ptr(ids), table.shape[0], table.shape[1],
            _ptr(table), float(scale), _ptr(out), _stream_ptr(stream, table.device))
    return _call(lib.embedding_nd, args, out, None, _prepare_only)


def embedding_backward_nd(dy: torch.Tensor, ids: torch.Tensor, rows: int, *, scale: float = 1.0,
                          padding_idx: Optional[int] = None, grad_dtype: Optional[torch.dtype] = None,
                          out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                          _prepare_only: bool = False) -> torch.Tensor:
    """The table's gradient (rows, width) of ``embedding_nd`` from y's gradient dy, of shape
    ids.shape + (width,), contiguous: the tokens sorted by id, each row's summed in float32
    in their order (the same bits every time).  ``padding_idx``: a row that takes no
    gradient.  ``grad_dtype``: dy's type (default) or float32."""
    lib = load_library()
    if dy.dtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, f"dtype {dy.dtype} is not served (float32, float16, bfloat16)")
    _check_tensor("dy", dy, dy.device, dy.dtype)
    _check_ids(ids, dy.device)
    if dy.dim() != ids.dim() + 1 or tuple(dy.shape[:-1]) != tuple(ids.shape) or not dy.is_contiguous():
        raise ConvTransposeError(1, "dy must be a dense tensor of shape ids.shape + (width,)")
    rows, width = int(rows), dy.shape[-1]
    if rows < 0:
        raise ConvTransposeError(1, "rows must not be negative")
    if padding_idx is not None and not 0 <= int(padding_idx) < rows:
        raise ConvTransposeError(1, "padding_idx must be a row of the table")
    grad_dtype = dy.dtype if grad_dtype is None else grad_dtype
    if grad_dtype not in (dy.dtype, torch.float32):
        raise ConvTransposeError(3, f"grad_dtype must be {dy.dtype} or float32 (got {grad_dtype})")
    if out is None:
        with _on(stream):
            out = torch.empty((rows, width), dtype=grad_dtype, device=dy.device)
    else:
        _check_tensor("out", out, dy.device, grad_dtype)
        if tuple(out.shape) != (rows, width) or not out.is_contiguous():
            raise ConvTransposeError(2, f"out must be dense with shape {(rows, width)}")
    nbytes = ctypes.c_size_t(0)
    if _prepare_only:
        st = lib.embedding_workspace_size(ids.numel(), rows, width, ctypes.byref(nbytes))
        if st:
            _raise(st)
    with _on(stream):
        ws, wsb = _scratch(nbytes.value, dy.device, _prepare_only)
    args = (_LAYER_DTYPES[dy.dtype], _INDEX_DTYPES[ids.dtype], ids.numel(), _ptr(ids), rows, width, _ptr(dy), float(scale),
            -1 if padding_idx is None else int(padding_idx), _LAYER_DTYPES[grad_dtype], _ptr(out), _ptr(ws), wsb,
            _stream_ptr(stream, dy.device))
    return _call(lib.embedding_backward_nd, args, out, ws, _prepare_only)


# ------------------------------------------------------------------------------------
# Attention over tokens, rotary positions, and the step that trains a model
# ------------------------------------------------------------------------------------
def _token_strides(name, t):
    """Strides of the image, token and head axes of an (N, T, H, D) tensor with dense heads."""
    if t.dim() != 4:
        raise ConvTransposeError(1, f"{name} must be (N, T, H, D)")
    if t.shape[3] > 1 and t.stride(3) != 1 and t.numel():
        raise ConvTransposeError(1, f"the elements of a head must be dense in {name}")
    return _i64(t.stride()[:3])


def _attention_args(q, k, v, scale, causal, lengths, starts):
    """Checks both directions of attention share; (sizes, operands, mask) arguments."""
    if q.dtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, f"dtype {q.dtype} is not served (float32, float16, bfloat16)")
    operands = []
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, q.device, q.dtype)
        operands += [_ptr(t), _token_strides(name, t)]
    if k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]:
        raise ConvTransposeError(1, "k and v must have one shape, and q's images and head size")
    if k.shape[2] < 1 or q.shape[2] < 1 or q.shape[2] % k.shape[2]:
        raise ConvTransposeError(1, "q's heads must be a multiple of k's")
    scale = q.shape[3] ** -0.5 if scale is None and q.shape[3] else scale
    if scale is None or not 0.0 < float(scale) <= 1e38:
        raise ConvTransposeError(1, "scale must lie in (0, 1e38]")
    if starts is not None and not causal:
        raise ConvTransposeError(1, "starts are for causal calls")
    for name, t in (("lengths", lengths), ("starts", starts)):
        if t is not None:
            _check_tensor(name, t, q.device, torch.int32)
            if tuple(t.shape) != (q.shape[0],) or not t.is_contiguous():
                raise ConvTransposeError(1, f"{name} must be a dense int32 tensor with one value an image")
    return ([_LAYER_DTYPES[q.dtype], _i64(q.shape), k.shape[1], k.shape[2]], operands,
            [float(scale), int(bool(causal)), _ptr(lengths), _ptr(starts)])


def _attention_workspace(sizes, backward):
    nbytes = ctypes.c_size_t(0)
    st = load_library().attention_workspace_size(*sizes, int(backward), ctypes.byref(nbytes))
    if st:
        _raise(st)
    return nbytes.value


def _dense_like(name, t, like):
    """A caller's output (None: a new one) of `like`'s shape and type, dense."""
    if t is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _check_tensor(name, t, like.device, like.dtype)
    if t.shape != like.shape or not t.is_contiguous():
        raise ConvTransposeError(2, f"{name} must be dense with shape {tuple(like.shape)}")
    return t


def attention_nd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: Optional[float] = None,
                 causal: bool = False, lengths: Optional[torch.Tensor] = None, starts: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                 _prepare_only: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out, lse): softmax(scale q k^T) v over tokens, and the logarithm of its denominators.

    q: (N, Tq, H, D) float32/float16/bfloat16; k, v: (N, Tk, Hkv, D), Hkv dividing H (head h reads key
    head h / (H / Hkv)); D up to 256, dense, the other axes with any strides: q, k and v may be
    parts of one projection, or a cache.  A channels-last (N, C, D1..Dn) tensor is
    ``x.movedim(1, -1).reshape(N, -1, H, C // H)``.  ``scale``: 1 / sqrt(D).  ``lengths``: (N,) int32,
    keys of each image (what stands behind them is never looked at).  ``causal``: query i sees
    the keys up to ``starts[n] + i``; ``starts``: (N,) int32, by default Tk - Tq.  A single token over a
    cache gives ``lengths`` with it and ``starts = lengths - 1``.  A query that sees nothing
    gives zeros and lse = -inf.  out is dense (N, Tq, H, D), lse (N, H, Tq) float32, for
    ``attention_backward_nd``."""
    lib = load_library()
    sizes, operands, mask = _attention_args(q, k, v, scale, causal, lengths, starts)
    nbytes = _attention_workspace(sizes, False) if _prepare_only else 0
    with _on(stream):
        if out is not None and out.numel() and out.data_ptr() in (q.data_ptr(), k.data_ptr(), v.data_ptr()):
            raise ConvTransposeError(1, "out must not be one of the inputs")
        out = _dense_like("out", out, q)
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
        ws, wsb = _scratch(nbytes, q.device, _prepare_only)
    args = (*sizes, *operands, *mask, _ptr(out), _ptr(lse), _ptr(ws), wsb, _stream_ptr(stream, q.device))
    return _call(lib.attention_nd, args, (out, lse), ws, _prepare_only)


def attention_backward_nd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                          lse: torch.Tensor, *, scale: Optional[float] = None, causal: bool = False,
                          lengths: Optional[torch.Tensor] = None, starts: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None, _prepare_only: bool = False
                          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv): the gradient of ``attention_nd`` from out's gradient dout, its inputs, and the out and
    lse it returned, with the same mask and scale.  dk and dv have k's shape: the query heads
    that share a key head are summed.  Dense results; the probabilities are computed again, and the
    sums have a fixed order."""
    lib = load_library()
    sizes, operands, mask = _attention_args(q, k, v, scale, causal, lengths, starts)
    for name, t in (("dout", dout), ("out", out)):
        _check_tensor(name, t, q.device, q.dtype)
        if t.shape != q.shape:
            raise ConvTransposeError(2, f"{name} has shape {tuple(t.shape)}, expected {tuple(q.shape)}")
    _check_tensor("lse", lse, q.device, torch.float32)
    if tuple(lse.shape) != (q.shape[0], q.shape[2], q.shape[1]) or not lse.is_contiguous():
        raise ConvTransposeError(1, "lse must be a dense (N, H, Tq) tensor")
    nbytes = _attention_workspace(sizes, True) if _prepare_only else 0
    with _on(stream):
        dq, dk, dv = (_dense_like(None, None, t) for t in (q, k, v))
        ws, wsb = _scratch(nbytes, q.device, _prepare_only)
    args = (*sizes, _ptr(dout), _token_strides("dout", dout), *operands, _ptr(out), _token_strides("out", out), _ptr(lse),
            *mask, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), wsb, _stream_ptr(stream, q.device))
    return _call(lib.attention_backward_nd, args, (dq, dk, dv), ws, _prepare_only)


def rotary_nd(x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int], *, base: float = 10000.0,
              whole_ladder: bool = False, interleaved: bool = False, inverse: bool = False,
              out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
              _prepare_only: bool = False) -> torch.Tensor:
    """Rotary positions with several axes: the first ``2 * sum(sections)`` elements of each head are pairs that
    turn by the token's positions, the rest is copied.

    x: (N, T, H, D) float32/float16/bfloat16, heads dense, the other axes with any strides, so the
    query and key heads of one projection turn in one call.  positions: (N, T, axes) int32/int64 (N and
    T may be expanded), for instance a token's time, height and width.  ``sections``: pairs of
    each axis; the j-th of a section of s turns ``base ** (-j / s)`` a position, or with
    ``whole_ladder`` the p-th of all R pairs ``base ** (-p / R)``.  A pair is (p, p + R), or (2 p, 2 p + 1)
    if ``interleaved``.  ``inverse`` turns back: the gradient of x is
    ``rotary_nd(dy, ..., inverse=True)``.  ``out``: the caller's y, which may be x."""
    lib = load_library()
    if x.dtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, f"dtype {x.dtype} is not served (float32, float16, bfloat16)")
    _check_tensor("x", x, x.device, x.dtype)
    strides = _token_strides("x", x)
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    if positions.dtype not in _INDEX_DTYPES:
        raise ConvTransposeError(3, f"positions must be int32 or int64 (got {positions.dtype})")
    _check_tensor("positions", positions, x.device, positions.dtype)
    axes = len(sections)
    if tuple(positions.shape) != (x.shape[0], x.shape[1], axes) or (axes > 1 and positions.stride(2) != 1):
        raise ConvTransposeError(1, "positions must be (N, T, axes) with one section an axis, its axes dense")
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _check_tensor("out", out, x.device, x.dtype)
        if out.shape != x.shape:
            raise ConvTransposeError(2, f"out has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
        if out.data_ptr() == x.data_ptr() and out.stride() != x.stride():
            raise ConvTransposeError(1, "out must have x's strides where it is x")
        if any(size > 1 and st == 0 for size, st in zip(out.shape, out.stride())):
            raise ConvTransposeError(1, "out must not be expanded")
    args = (_LAYER_DTYPES[x.dtype], _i64(x.shape), _ptr(x), strides, _INDEX_DTYPES[positions.dtype], axes, _ptr(positions),
            _i64(positions.stride()[:2]), _i64(sections), float(base), int(bool(whole_ladder)), int(bool(interleaved)),
            int(bool(inverse)), _ptr(out), _token_strides("out", out), _stream_ptr(stream, x.device))
    return _call(lib.rotary_nd, args, out, None, _prepare_only)


class _AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_scale", "v_scale", "copy")] + [
        ("count", ctypes.c_int64), ("weight_decay", ctypes.c_float)]


def _device_scalar(name, value, dtype, device):
    """(host value, pointer) of a number or of a one-element device tensor."""
    if not isinstance(value, torch.Tensor):
        return value, None
    _check_tensor(name, value, device, dtype)
    if value.numel() != 1:
        raise ConvTransposeError(1, f"{name} must hold one value")
    return 1, _ptr(value)


def adamw_nd(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], ms: Sequence[torch.Tensor],
             vs: Sequence[torch.Tensor], *, lr, step, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
             weight_decay=0.01, grad_scale=1.0, m_scales: Optional[Sequence[torch.Tensor]] = None,
             v_scales: Optional[Sequence[torch.Tensor]] = None, copies: Optional[Sequence[Optional[torch.Tensor]]] = None,
             stream: Optional[torch.cuda.Stream] = None, _prepare_only: bool = False) -> Tuple[torch.Tensor, ...]:
    """One AdamW step over all ``params``, in place; returns them.

    params: float32/float16/bfloat16, grads: any of these, all dense and of one type each.  ms, vs: the
    moments, float32; or float8_e4m3fn with ``m_scales`` and ``v_scales``, a float32 for each 256
    consecutive elements (m = value * scale, sqrt(v) = value * scale), all zeros at the start.  8 bits are for
    ``betas[1]`` up to 0.95: at 0.99 and more a second moment that falls beside others of its 256 does not
    follow, since a step changes it by less than half a code.
    ``step``: the number of the step, from 1.  ``weight_decay``: one number, or one a tensor.
    ``grad_scale``: multiplies the gradients (one over a loss scale).  ``copies``: float16 or bfloat16
    tensors (or None) that receive the updated parameters too.  ``lr``, ``step`` and ``grad_scale`` may be
    one-element device tensors (float32, int64, float32), read when the kernel runs, so a captured or
    prepared call follows them."""
    lib = load_library()
    params, count = tuple(params), len(params)
    lists = [("grads", grads), ("ms", ms), ("vs", vs)]
    lists += [(n, t) for n, t in (("m_scales", m_scales), ("v_scales", v_scales), ("copies", copies)) if t is not None]
    for name, t in lists:
        if len(t) != count:
            raise ConvTransposeError(1, f"{name} must hold one tensor a parameter")
    decay = [float(weight_decay)] * count if not hasattr(weight_decay, "__len__") else [float(w) for w in weight_decay]
    if len(decay) != count:
        raise ConvTransposeError(1, "weight_decay must be one number, or one a parameter")
    if not count:
        if _prepare_only:
            raise ConvTransposeError(1, "there are no parameters")
        return params
    dev, dtype, gtype, stype = params[0].device, params[0].dtype, grads[0].dtype, ms[0].dtype
    if dtype not in _LAYER_DTYPES or gtype not in _LAYER_DTYPES:
        raise ConvTransposeError(3, "params and grads must be float32, float16 or bfloat16")
    if stype not in (torch.float32, torch.float8_e4m3fn):
        raise ConvTransposeError(3, f"the moments must be float32 or float8_e4m3fn (got {stype})")
    bits = 32 if stype == torch.float32 else 8
    if (bits == 8) != (m_scales is not None) or (bits == 8) != (v_scales is not None):
        raise ConvTransposeError(1, "m_scales and v_scales belong to moments in float8_e4m3fn")
    written = [c for c in copies or () if c is not None]
    ctype = written[0].dtype if written else torch.float16
    if ctype not in (torch.float16, torch.bfloat16):
        raise ConvTransposeError(3, f"copies must be float16 or bfloat16 (got {ctype})")
    table, seen = (_AdamWTensor * count)(), set()
    for i in range(count):
        n = params[i].numel()
        parts = [("params", params[i], dtype, n), ("grads", grads[i], gtype, n), ("ms", ms[i], stype, n), ("vs", vs[i], stype, n)]
        for name, scales in (("m_scales", m_scales), ("v_scales", v_scales)):
            parts.append((name, None if scales is None else scales[i], torch.float32, (n + 255) // 256))
        parts.append(("copies", copies[i] if copies is not None else None, ctype, n))
        for name, t, kind, size in parts:
            if t is None:
                continue
            _check_tensor(name, t, dev, kind)
            if t.numel() != size or not t.is_contiguous():
                raise ConvTransposeError(1, f"{name}[{i}] must be dense with {size} elements")
            if name != "grads" and size:
                if t.data_ptr() in seen:
                    raise ConvTransposeError(1, f"{name}[{i}] is there twice")
                seen.add(t.data_ptr())
        table[i] = _AdamWTensor(*(None if t is None else t.data_ptr() for _, t, _, _ in parts), n, decay[i])
    lr, lr_at = _device_scalar("lr", lr, torch.float32, dev)
    step, step_at = _device_scalar("step", step, torch.int64, dev)
    grad_scale, scale_at = _device_scalar("grad_scale", grad_scale, torch.float32, dev)
    args = (_LAYER_DTYPES[dtype], _LAYER_DTYPES[gtype], bits, _LAYER_DTYPES[ctype], count, table, float(lr), lr_at,
            float(betas[0]), float(betas[1]), float(eps), int(step), step_at, float(grad_scale), scale_at,
            _stream_ptr(stream, dev))
    return _call(lib.adamw_nd, args, params, None, _prepare_only)


class PreparedCall:
    """One call of ``convolution_nd``, ``qlinear_convtranspose_nd``, ``group_norm_nd``,
    ``group_norm_backward_nd``, ``dropout_nd``, ``embedding_nd``, ``embedding_backward_nd``,
    ``attention_nd``, ``attention_backward_nd``, ``rotary_nd`` or ``adamw_nd`` with its
    arguments validated and marshalled once (and its workspace, where it takes one,
    allocated): ``PreparedCall(convolution_nd, x, w, ...)``
    takes the function's own arguments; each call then enqueues the operation with a single
    C call, writing the same output tensors (``.out``).  Repeated calls must be ordered on
    one stream; the tensors must outlive the object."""

    def __init__(self, fn, *args, **kwargs):
        if fn not in (convolution_nd, qlinear_convtranspose_nd, group_norm_nd, group_norm_backward_nd, dropout_nd,
                      embedding_nd, embedding_backward_nd, attention_nd, attention_backward_nd, rotary_nd, adamw_nd):
            raise TypeError("PreparedCall serves the package's functions that take tensors and return new ones, "
                            "except convtranspose_nd (ConvTransposePlan)")
        self._fn, self._args, self.out, *keep = fn(*args, _prepare_only=True, **kwargs)
        self._keep = (args, kwargs, keep)  # the pointers stay valid while the object lives
        self.device = (self.out[0] if isinstance(self.out, tuple) else self.out).device

    def __call__(self) -> torch.Tensor:
        if torch.cuda.current_device() == self.device.index:  # entering the device costs a microsecond
            st = self._fn(*self._args)
        else:
            with torch.cuda.device(self.device):
                st = self._fn(*self._args)
        if st:
            _raise(st)
        return self.out
