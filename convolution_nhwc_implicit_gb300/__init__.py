"""Python binding of the fused NHWC convolution library (``libconv_nhwc.so``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
fallback: if the compiled library is missing or cannot be loaded, importing
this package raises.

Names follow the C ABI in ``include/conv_nhwc.h``::

    plan = Plan(n, h, w, c_in, c_out, k_h, k_w, stride=1, pad_h=0, pad_w=0,
                groups=1, dtype="bf16", act="mish", quant=None)
    plan.run(x, w, b, y)          # torch CUDA tensors, NHWC / OHWI layouts
    y = conv2d_nhwc(x, w, b, stride=..., pad=(ph, pw), act="mish")
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from array import array

__all__ = ["Plan", "ConvError", "conv2d_nhwc", "library_path", "load_library", "DTYPES", "ACTS",
           "ALGOS", "status_str", "abi_version", "run_i8_noalloc", "NOALLOC_MAX_COUT", "spp", "DwpwPlan",
           "GroupNormPlan", "ClassLossPlan", "W4Plan", "w4_quantize", "BlockNormPlan", "GradClipPlan", "NORMS"]

# Largest c_out conv_run_i8_noalloc accepts (its fixed scratch array holds
# that many requantisation multipliers).
NOALLOC_MAX_COUT = 4096

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libconv_nhwc.so")

DTYPES = {"f32": 0, "bf16": 1, "i8": 2}
ACTS = {"none": 0, "relu": 1, "mish": 2}
NORMS = {"none": 0, "layer": 1, "rms": 2}
ALGOS = {"auto": 0, "direct": 1, "depthwise": 2, "igemm": 3, "igemm_swapped": 4, "igemm_n256": 5,
         "igemm_n128": 6, "igemm_n64": 7, "igemm_pair": 8, "dwpw": 9, "igemm_pair128": 10,
         "groupnorm": 11, "w4": 12, "xent": 13, "blocknorm": 14, "gradclip": 15}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
# Staging, epilogue and int8-widening flags of the tensor-core family
# (CONV_ALGO_STAGE_*, CONV_ALGO_EPI_*, CONV_ALGO_WIDEN_*), written as suffixes
# of the algo name: "igemm+halo", "igemm_n64+taps+ept", "igemm+inkernel".
ALGO_FLAGS = {"taps": 0x100, "halo": 0x200, "sliced": 0x400, "ept": 0x800, "prepass": 0x1000,
              "inkernel": 0x2000}


def _algo_code(algo: str) -> int:
    name, *flags = algo.split("+")
    code = ALGOS[name]
    for f in flags:
        code |= ALGO_FLAGS[f]
    return code


class ConvError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {status_str(code)} ({code})")
        self.code = code


class _Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "h", "w", "c_in", "c_out", "k_h", "k_w")]


class _Output(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("y_channels", "y_channel_offset", "upsample", "residual")]


class _Quant(ctypes.Structure):
    _fields_ = [("in_scale", ctypes.c_float), ("out_scale", ctypes.c_float),
                ("w_scales", ctypes.POINTER(ctypes.c_float))]


class _BlockNormPointers(ctypes.Structure):
    """conv_blocknorm_params_t and conv_blocknorm_grads_t."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("scale", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta")]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Loads libconv_nhwc.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -m convolution_nhwc_implicit_gb300.build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(_LIB_PATH)
    c_int, c_void_p, pp = ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)
    lib.conv_plan_create.argtypes = [ctypes.POINTER(_Shape), c_int, c_int, c_int, c_int, c_int, c_int,
                                     ctypes.POINTER(_Quant), pp]
    lib.conv_plan_create.restype = c_int
    lib.conv_plan_create_ex.argtypes = [ctypes.POINTER(_Shape), c_int, c_int, c_int, c_int, c_int, c_int,
                                        ctypes.POINTER(_Quant), c_int, pp]
    lib.conv_plan_create_ex.restype = c_int
    lib.conv_plan_create_fused.argtypes = [ctypes.POINTER(_Shape), c_int, c_int, c_int, c_int, c_int, c_int,
                                           ctypes.POINTER(_Quant), ctypes.POINTER(_Output), c_int, pp]
    lib.conv_plan_create_fused.restype = c_int
    lib.conv_run.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.conv_run.restype = c_int
    lib.conv_run_fused.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.conv_run_fused.restype = c_int
    lib.conv_plan_destroy.argtypes = [c_void_p]
    lib.conv_plan_destroy.restype = None
    lib.conv_plan_output_shape.argtypes = [c_void_p, ctypes.POINTER(c_int), ctypes.POINTER(c_int)]
    lib.conv_plan_output_shape.restype = c_int
    lib.conv_plan_algo.argtypes = [c_void_p]
    lib.conv_plan_algo.restype = c_int
    lib.conv_plan_launches.argtypes = [c_void_p]
    lib.conv_plan_launches.restype = c_int
    lib.conv_plan_describe.argtypes = [c_void_p]
    lib.conv_plan_describe.restype = ctypes.c_char_p
    lib.conv_plan_check_device_status.argtypes = [c_void_p, c_void_p]
    lib.conv_plan_check_device_status.restype = c_int
    lib.conv_status_str.argtypes = [c_int]
    lib.conv_status_str.restype = ctypes.c_char_p
    lib.conv_abi_version.argtypes = []
    lib.conv_abi_version.restype = c_int
    lib.conv_run_i8_noalloc.argtypes = [ctypes.POINTER(_Shape), c_int, c_int, c_int, c_int, c_int,
                                        ctypes.POINTER(_Quant), c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p]
    lib.conv_run_i8_noalloc.restype = c_int
    lib.conv_plan_create_dwpw.argtypes = [ctypes.POINTER(_Shape), c_int, c_int, c_int, c_int, c_int, pp]
    lib.conv_plan_create_dwpw.restype = c_int
    lib.conv_run_dwpw.argtypes = [c_void_p] * 8
    lib.conv_run_dwpw.restype = c_int
    lib.conv_spp_run.argtypes = [c_int, c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                 c_int, c_void_p]
    lib.conv_spp_run.restype = c_int
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    for name, args in (
            ("conv_plan_workspace", [c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
            ("conv_plan_workspace_bwd", [c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
            ("conv_plan_create_groupnorm", [i32, i32, i32, i32, i32, ctypes.c_float, c_int, c_int, pp]),
            ("conv_run_groupnorm", [c_void_p, c_void_p, i64, c_void_p, c_void_p, c_void_p, i64] + [c_void_p] * 4),
            ("conv_run_groupnorm_bwd", [c_void_p, c_void_p, i64] + [c_void_p] * 4 + [c_void_p, i64, c_void_p, i64] +
             [c_void_p] * 4),
            ("conv_plan_create_xent", [i32, i32, i32, i32, c_int, pp]),
            ("conv_run_xent", [c_void_p] * 9),
            ("conv_run_xent_bwd", [c_void_p] * 10),
            ("conv_plan_create_w4", [i32, i32, i32, i32, c_int, c_int, pp]),
            ("conv_w4_packed_bytes", [i32, i32, ctypes.POINTER(ctypes.c_size_t)]),
            ("conv_w4_pack", [i32, i32, c_void_p, c_void_p, c_void_p]),
            ("conv_w4_quantize", [i32, i32, i32, c_int] + [c_void_p] * 4),
            ("conv_run_w4", [c_void_p] * 7),
            ("conv_plan_create_blocknorm", [i32, i32, i32, i32, c_int, c_int, ctypes.c_float, c_int, pp]),
            ("conv_run_blocknorm", [c_void_p, c_void_p, i64, c_void_p, i64, ctypes.POINTER(_BlockNormPointers), c_void_p, i64,
                                    c_void_p, i64, c_void_p, c_void_p]),
            ("conv_run_blocknorm_bwd", [c_void_p, c_void_p, i64, c_void_p, i64, ctypes.POINTER(_BlockNormPointers), c_void_p] +
             [c_void_p, i64] * 4 + [ctypes.POINTER(_BlockNormPointers), c_void_p, c_void_p]),
            ("conv_plan_create_gradclip", [i32, ctypes.POINTER(i64), ctypes.POINTER(c_int), pp]),
            ("conv_run_gradclip", [c_void_p, c_void_p, c_void_p, ctypes.c_float, c_void_p, c_void_p, c_void_p])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def status_str(code: int) -> str:
    return load_library().conv_status_str(int(code)).decode()


def abi_version() -> int:
    return load_library().conv_abi_version()


def _ptr(t):
    """Device pointer of a torch tensor (or None / an int address)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_cuda = None


def _cuda_getters():
    """Torch's getters of the current device and of the handle of a device's
    current stream, looked up once (the raw forms spare a small call the 3 us of
    building a Stream object)."""
    global _cuda
    if _cuda is None:
        import torch
        try:
            _cuda = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        except AttributeError:
            _cuda = torch.cuda.current_device, lambda device: torch.cuda.current_stream(device).cuda_stream
    return _cuda


def _current_device():
    return (_cuda or _cuda_getters())[0]()


def _current_stream(device=None):
    """Handle of torch's current stream (on `device`, if the caller knows the current one)."""
    device_of, stream_of = _cuda_getters()
    return stream_of(device_of() if device is None else device)


_raw_memory = None


def _raw_memory_calls():
    """Torch's allocator without a tensor around the block: an address of a
    stream's memory, and its return.  A run's scratch is a block of the run's own
    stream, given back when the run is queued: whoever gets it next is ordered
    after the run.  Looked up once.  (Among launches a tensor costs a call 5 us,
    this 1.5.)"""
    global _raw_memory
    if _raw_memory is None:
        import torch
        torch.cuda.init()
        try:
            _raw_memory = torch._C._cuda_cudaCachingAllocator_raw_alloc, torch._C._cuda_cudaCachingAllocator_raw_delete
        except AttributeError:
            def alloc(nbytes, handle):
                return torch.cuda.caching_allocator_alloc(nbytes, stream=handle)
            _raw_memory = alloc, torch.cuda.caching_allocator_delete
    return _raw_memory


def _stream_handle(stream, device=None):
    if stream is None:
        return _current_stream(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _allocating_on(stream, device):
    """A context in which torch's allocator hands out blocks of `stream` (None:
    the current one).  A block of another stream may still be in use by kernels
    queued there, whatever it is told afterwards."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class Plan:
    """A validated layer bound to the current CUDA device (see conv_plan_create).

    ``out`` (optional) holds the output options of conv_plan_create_fused:
    dict(y_channels=0, y_channel_offset=0, upsample=1, residual=False)."""

    def __init__(self, n, h, w, c_in, c_out, k_h, k_w, stride=1, pad_h=0, pad_w=0, groups=1,
                 dtype="bf16", act="none", quant=None, algo="auto", out=None):
        lib = load_library()
        self._lib = lib
        self._handle = ctypes.c_void_p()
        self.shape = (n, h, w, c_in, c_out, k_h, k_w)
        self.stride, self.pad_h, self.pad_w, self.groups = stride, pad_h, pad_w, groups
        self.dtype, self.act = dtype, act
        shape = _Shape(n, h, w, c_in, c_out, k_h, k_w)
        qp = None
        if quant is not None:
            in_scale, out_scale, w_scales = quant
            ws = [float(v) for v in w_scales]
            self._ws = (ctypes.c_float * len(ws))(*ws)
            qp = ctypes.pointer(_Quant(float(in_scale), float(out_scale),
                                       ctypes.cast(self._ws, ctypes.POINTER(ctypes.c_float))))
        op = None
        self.out = dict(y_channels=c_out, y_channel_offset=0, upsample=1, residual=False)
        if out is not None:
            o = dict(self.out, **out)
            o["y_channels"] = o["y_channels"] or c_out
            self.out = o
            op = ctypes.pointer(_Output(int(o["y_channels"]), int(o["y_channel_offset"]), int(o["upsample"]),
                                        int(bool(o["residual"]))))
        rc = lib.conv_plan_create_fused(ctypes.byref(shape), stride, pad_h, pad_w, groups, DTYPES[dtype],
                                        ACTS[act], qp, op, _algo_code(algo), ctypes.byref(self._handle))
        if rc != 0:
            raise ConvError("conv_plan_create", rc)
        oh, ow = ctypes.c_int(), ctypes.c_int()
        lib.conv_plan_output_shape(self._handle, ctypes.byref(oh), ctypes.byref(ow))
        self.oh, self.ow = oh.value, ow.value

    @property
    def handle(self) -> int:
        return self._handle.value

    @property
    def output_shape(self):
        """Shape of the layer's own output [N, OH, OW, Cout]."""
        n, _, _, _, c_out, _, _ = self.shape
        return (n, self.oh, self.ow, c_out)

    @property
    def y_shape(self):
        """Shape of the y buffer the plan writes into (with its output options)."""
        u = self.out["upsample"]
        return (self.shape[0], self.oh * u, self.ow * u, self.out["y_channels"])

    @property
    def algo(self) -> str:
        return ALGO_NAMES[self._lib.conv_plan_algo(self._handle)]

    @property
    def launches(self) -> int:
        """Kernels one run() enqueues."""
        return self._lib.conv_plan_launches(self._handle)

    def describe(self) -> str:
        return self._lib.conv_plan_describe(self._handle).decode()

    def run(self, x, w, b, y, stream=None, residual=None) -> None:
        """Enqueue y = act(conv(x, w) + b) [+ residual] on `stream` (default: torch's current stream)."""
        if residual is None:
            rc = self._lib.conv_run(self._handle, _ptr(x), _ptr(w), _ptr(b), _ptr(y), _stream_handle(stream))
        else:
            rc = self._lib.conv_run_fused(self._handle, _ptr(x), _ptr(w), _ptr(b), _ptr(residual), _ptr(y),
                                          _stream_handle(stream))
        if rc != 0:
            raise ConvError("conv_run", rc)

    def check_device_status(self, stream=None) -> None:
        rc = self._lib.conv_plan_check_device_status(self._handle, _stream_handle(stream))
        if rc != 0:
            raise ConvError("conv_plan_check_device_status", rc)

    def close(self) -> None:
        if getattr(self, "_handle", None) is not None and self._handle.value:
            self._lib.conv_plan_destroy(self._handle)
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def conv2d_nhwc(x, w, b=None, stride=1, pad=(0, 0), groups=1, act="none", quant=None, algo="auto",
                plan=None, out=None):
    """One-shot helper on torch CUDA tensors: x NHWC, w OHWI, b [Cout].

    Builds a plan (unless given), allocates y with torch (unless ``out``) and
    runs the layer on the current stream."""
    import torch
    dt = {torch.float32: "f32", torch.bfloat16: "bf16", torch.int8: "i8"}[x.dtype]
    n, h, wd, c_in = x.shape
    c_out, k_h, k_w, _ = w.shape
    if plan is None:
        plan = Plan(n, h, wd, c_in, c_out, k_h, k_w, stride, pad[0], pad[1], groups, dt, act, quant, algo)
    if out is None:
        out = torch.empty(plan.output_shape, dtype=x.dtype, device=x.device)
    plan.run(x, w, b, out)
    return out


def run_i8_noalloc(x, w, b, y, stride=1, pad=(0, 0), groups=1, act="none", quant=None, stream=None):
    """An int8 layer through conv_run_i8_noalloc: no plan and no device
    allocation, for callers that must not allocate device memory at run time
    (their buffers come from a pre-reserved pool).  The library keeps the
    requantisation table in one fixed device array shared by all calls, so
    calls that may overlap on the GPU must be serialised.  x NHWC, w OHWI,
    b int32 [Cout] or None, y preallocated NHWC int8; quant = (s_x, s_y, s_w)."""
    lib = load_library()
    n, h, wd, c_in = x.shape
    c_out, k_h, k_w, _ = w.shape
    in_scale, out_scale, w_scales = quant
    ws = (ctypes.c_float * c_out)(*[float(v) for v in w_scales])
    q = _Quant(float(in_scale), float(out_scale), ctypes.cast(ws, ctypes.POINTER(ctypes.c_float)))
    shape = _Shape(n, h, wd, c_in, c_out, k_h, k_w)
    rc = lib.conv_run_i8_noalloc(ctypes.byref(shape), stride, pad[0], pad[1], groups, ACTS[act],
                                 ctypes.byref(q), _ptr(x), _ptr(w), _ptr(b), _ptr(y), _stream_handle(stream))
    if rc != 0:
        raise ConvError("conv_run_i8_noalloc", rc)
    return y


def spp(x, y, y_channels=None, off5=None, off9=None, off13=None, off_x=-1, stream=None):
    """SPP block (conv_spp_run): the 5x5, 9x9 and 13x13 max pools of x (NHWC,
    torch CUDA tensor) written into channel slices of y.  Defaults: y has
    4*C channels laid out [mp5 | mp9 | mp13 | x]."""
    n, h, w, c = x.shape
    y_channels = y_channels or 4 * c
    off5 = 0 if off5 is None else off5
    off9 = c if off9 is None else off9
    off13 = 2 * c if off13 is None else off13
    if off_x is None:
        off_x = 3 * c
    dt = {"torch.float32": 0, "torch.bfloat16": 1, "torch.int8": 2}[str(x.dtype)]
    rc = load_library().conv_spp_run(n, h, w, c, dt, _ptr(x), _ptr(y), y_channels, off5, off9, off13, off_x,
                                     _stream_handle(stream))
    if rc != 0:
        raise ConvError("conv_spp_run", rc)


class DwpwPlan(Plan):
    """A fused depthwise 3x3 -> pointwise 1x1 pair (conv_plan_create_dwpw):
    y = act_pw(pw(round(act_dw(dw(x) + b_dw))) + b_pw), the intermediate kept
    on chip."""

    def __init__(self, n, h, w, c, c_out, stride=1, pad=1, dtype="f32", act_dw="relu", act_pw="relu"):
        lib = load_library()
        self._lib = lib
        self._handle = ctypes.c_void_p()
        self.shape = (n, h, w, c, c_out, 3, 3)
        self.stride, self.pad_h, self.pad_w, self.groups = stride, pad, pad, 1
        self.dtype, self.act, self.act_pw = dtype, act_dw, act_pw
        self.out = dict(y_channels=c_out, y_channel_offset=0, upsample=1, residual=False)
        shape = _Shape(n, h, w, c, c_out, 3, 3)
        rc = lib.conv_plan_create_dwpw(ctypes.byref(shape), stride, pad, DTYPES[dtype], ACTS[act_dw], ACTS[act_pw],
                                       ctypes.byref(self._handle))
        if rc != 0:
            raise ConvError("conv_plan_create_dwpw", rc)
        oh, ow = ctypes.c_int(), ctypes.c_int()
        lib.conv_plan_output_shape(self._handle, ctypes.byref(oh), ctypes.byref(ow))
        self.oh, self.ow = oh.value, ow.value

    def run(self, x, w_dw, b_dw, w_pw, b_pw, y, stream=None) -> None:  # noqa: D401
        """Enqueue the fused pair on `stream` (default: torch's current stream)."""
        rc = self._lib.conv_run_dwpw(self._handle, _ptr(x), _ptr(w_dw), _ptr(b_dw), _ptr(w_pw), _ptr(b_pw),
                                     _ptr(y), _stream_handle(stream))
        if rc != 0:
            raise ConvError("conv_run_dwpw", rc)


def _dtype_name(t) -> str:
    name = {"torch.float32": "f32", "torch.bfloat16": "bf16", "torch.int8": "i8"}.get(str(t.dtype))
    if name is None:
        raise TypeError(f"tensors of {t.dtype} are not supported")
    return name


def _check(name, t, shape, dtype, device):
    """Checks a dense tensor argument on CUDA device `device` and returns its device pointer."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on cuda:{device}, got one on {t.device}")
    return t.data_ptr()


_getters = None


def _tensor_getters():
    """What is asked of every tensor of a call, to be mapped over all of them
    (about 0.04 us each, where a loop takes twice that): its shape, dtype,
    whether it is dense, its device, its address and its number of elements.
    Looked up once."""
    global _getters
    if _getters is None:
        import operator

        import torch
        t = torch.Tensor
        _getters = (operator.attrgetter("shape"), operator.attrgetter("dtype"), t.is_contiguous, t.get_device, t.data_ptr,
                    t.numel)
    return _getters


def _torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "u8": torch.uint8, "i32": torch.int32}[name]


class _OpPlan(Plan):
    """What the plans of the operators around the layer share.  A plan belongs
    to the device that is current when it is made; its runs take tensors of that
    device, with it current."""

    def _create(self, fn, *args):
        self._lib = load_library()
        self._handle = ctypes.c_void_p()
        rc = getattr(self._lib, fn)(*args, ctypes.byref(self._handle))
        if rc != 0:
            raise ConvError(fn, rc)
        self._device = _current_device()
        n = ctypes.c_size_t()
        self._lib.conv_plan_workspace(self._handle, ctypes.byref(n))
        self.workspace_bytes = n.value
        self._lib.conv_plan_workspace_bwd(self._handle, ctypes.byref(n))
        self.workspace_bytes_backward = n.value
        self._f32, self._dt = _torch_dtype("f32"), _torch_dtype(self.dtype)

    def _on_device(self):
        """The plan's device, which a run needs to be the current one."""
        now = _current_device()
        if now != self._device:
            raise ValueError(f"the plan belongs to cuda:{self._device}, and cuda:{now} is current")
        return now

    def _workspace(self, nbytes, like, stream):
        """Scratch of one run, a block of the run's own stream: whoever gets it
        next from torch's allocator is ordered after the run."""
        if not nbytes:
            return None
        import torch
        if stream is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        with _allocating_on(stream, like.device):
            return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


class _MapPlan(_OpPlan):
    """Plans whose runs take feature maps [n, h, w, c], ``shape``, dense or
    channel slices of a wider dense buffer (``buf[..., a:a + c]``)."""

    def _map(self, name, t):
        """Pointer and pixel pitch of a feature map."""
        n, h, w, c = self.shape
        if t is None:
            raise ValueError(f"{name} is missing")
        if t.dtype is not self._dt:
            raise TypeError(f"{name} is {t.dtype}, expected {self._dt}")
        if t.shape != self.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {self.shape}")
        if t.get_device() != self._device:
            raise ValueError(f"{name} must be on cuda:{self._device}, got a tensor on {t.device}")
        return t.data_ptr(), c if t.is_contiguous() else self._pitch(name, t)

    def _pitch(self, name, t):
        """Pixel pitch of a feature map that is not dense."""
        n, h, w, c = self.shape
        sn, sh, sw, sc = t.stride()
        # a size of one says nothing about its stride
        pitch = sw if w > 1 else (sh if h > 1 else (sn if n > 1 else c))
        if ((c > 1 and sc != 1) or pitch < c or (h > 1 and sh != w * pitch) or (n > 1 and sn != h * w * pitch)):
            raise ValueError(f"{name}: pixels must lie one pitch apart with their channels together, got strides {t.stride()}")
        return pitch


class GroupNormPlan(_MapPlan):
    """Group norm with an activation over NHWC maps (conv_plan_create_groupnorm).

    x, y, dy and dx are [n, h, w, c] CUDA tensors, dense or channel slices of a
    wider dense buffer (``buf[..., a:a + c]``); gamma, beta, dgamma and dbeta
    float32 [c]; mean and rstd float32 [n, groups]."""

    def __init__(self, n, h, w, c, groups, eps=1e-5, dtype="bf16", act="none"):
        self.shape = (n, h, w, c)
        self.groups, self.eps, self.dtype, self.act = groups, eps, dtype, act
        self._create("conv_plan_create_groupnorm", n, h, w, c, groups, float(eps), DTYPES[dtype], ACTS[act])
        self._cshape, self._sshape = (c,), (n, groups)

    @property
    def output_shape(self):
        return self.shape

    y_shape = output_shape

    def run(self, x, gamma, beta, y, mean=None, rstd=None, stream=None) -> None:  # noqa: D401
        """Enqueue y = act(group_norm(x) * gamma + beta) on `stream` (default: torch's current stream)."""
        f32, cs, ss, dev = self._f32, self._cshape, self._sshape, self._on_device()
        (px, pitch_x), (py, pitch_y) = self._map("x", x), self._map("y", y)
        g = None if gamma is None else _check("gamma", gamma, cs, f32, dev)
        b = None if beta is None else _check("beta", beta, cs, f32, dev)
        m = None if mean is None else _check("mean", mean, ss, f32, dev)
        r = None if rstd is None else _check("rstd", rstd, ss, f32, dev)
        ws = self._workspace(self.workspace_bytes, x, stream)
        rc = self._lib.conv_run_groupnorm(self._handle, px, pitch_x, g, b, py, pitch_y, m, r, _ptr(ws),
                                          _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_run_groupnorm", rc)

    def run_backward(self, x, gamma, beta, mean, rstd, dy, dx, dgamma=None, dbeta=None, stream=None) -> None:
        """Enqueue the gradient: dx, and dgamma and dbeta where given."""
        f32, cs, ss, dev = self._f32, self._cshape, self._sshape, self._on_device()
        (px, pitch_x), (pdy, pitch_dy), (pdx, pitch_dx) = self._map("x", x), self._map("dy", dy), self._map("dx", dx)
        g = None if gamma is None else _check("gamma", gamma, cs, f32, dev)
        b = None if beta is None else _check("beta", beta, cs, f32, dev)
        m, r = _check("mean", mean, ss, f32, dev), _check("rstd", rstd, ss, f32, dev)
        dg = None if dgamma is None else _check("dgamma", dgamma, cs, f32, dev)
        db = None if dbeta is None else _check("dbeta", dbeta, cs, f32, dev)
        ws = self._workspace(self.workspace_bytes_backward, x, stream)
        rc = self._lib.conv_run_groupnorm_bwd(self._handle, px, pitch_x, g, b, m, r, pdy, pitch_dy, pdx, pitch_dx, dg, db,
                                              _ptr(ws), _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_run_groupnorm_bwd", rc)


class ClassLossPlan(_OpPlan):
    """Softmax cross entropy of a class head over many classes, and its gradient
    (conv_plan_create_xent): scores x w^T that are never stored.

    x [rows, c_in] and w [classes, c_in] bf16; target int32 [rows], a row whose
    target is no class is left out; the loss is the mean over the others.
    ``piece`` bounds the classes the gradient works on at a time (0: chosen)."""

    def __init__(self, rows, c_in, classes, piece=0, dtype="bf16"):
        self.shape = (rows, c_in, classes)
        self.dtype, self.act = dtype, "none"
        self._create("conv_plan_create_xent", rows, c_in, classes, piece, DTYPES[dtype])
        self._i32 = _torch_dtype("i32")

    @property
    def output_shape(self):
        return ()

    y_shape = output_shape

    def run(self, x, w, target, loss, lse=None, row_loss=None, stream=None) -> None:  # noqa: D401
        """Enqueue the loss (a float32 scalar) and, where given, lse and row_loss (float32 [rows])."""
        rows, c_in, classes = self.shape
        f32, bf16, dev = self._f32, self._dt, self._on_device()
        px, pw = _check("x", x, (rows, c_in), bf16, dev), _check("w", w, (classes, c_in), bf16, dev)
        pt, pl = _check("target", target, (rows,), self._i32, dev), _check("loss", loss, (), f32, dev)
        ps = None if lse is None else _check("lse", lse, (rows,), f32, dev)
        pr = None if row_loss is None else _check("row_loss", row_loss, (rows,), f32, dev)
        ws = self._workspace(self.workspace_bytes, x, stream)
        rc = self._lib.conv_run_xent(self._handle, px, pw, pt, pl, pr, ps, _ptr(ws), _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_run_xent", rc)

    def run_backward(self, x, w, target, lse, dx, dw, dloss=None, stream=None) -> None:
        """Enqueue the gradient of the loss times dloss (a float32 scalar tensor; None: 1)."""
        rows, c_in, classes = self.shape
        f32, bf16, dev = self._f32, self._dt, self._on_device()
        px, pw = _check("x", x, (rows, c_in), bf16, dev), _check("w", w, (classes, c_in), bf16, dev)
        pt, ps = _check("target", target, (rows,), self._i32, dev), _check("lse", lse, (rows,), f32, dev)
        pdx, pdw = _check("dx", dx, (rows, c_in), bf16, dev), _check("dw", dw, (classes, c_in), bf16, dev)
        pd = None if dloss is None else _check("dloss", dloss, (), f32, dev)
        ws = self._workspace(self.workspace_bytes_backward, x, stream)
        rc = self._lib.conv_run_xent_bwd(self._handle, px, pw, pt, ps, pd, pdx, pdw, _ptr(ws), _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_run_xent_bwd", rc)


class W4Plan(_OpPlan):
    """Pointwise layer on few rows with 4-bit weights and group scales
    (conv_plan_create_w4): y = act(x W^T + bias), W = (code - 8) * scale.

    codes: uint8 [c_out, ceil(c_in / 2)], laid out once by ``pack``; scales
    [c_out, ceil(c_in / group)] of the plan's dtype; bias float32 [c_out] or
    None; x [rows, c_in] and y [rows, c_out] dense."""

    def __init__(self, rows, c_in, c_out, group=128, dtype="bf16", act="none"):
        self.shape = (rows, c_in, c_out)
        self.group, self.dtype, self.act = group, dtype, act
        self._create("conv_plan_create_w4", rows, c_in, c_out, group, DTYPES[dtype], ACTS[act])
        n = ctypes.c_size_t()
        self._lib.conv_w4_packed_bytes(c_in, c_out, ctypes.byref(n))
        self.packed_bytes = n.value
        self._u8 = _torch_dtype("u8")
        self._shapes = (rows, c_in), (self.packed_bytes,), (c_out, -(-c_in // group)), (c_out,), (rows, c_out)

    @property
    def output_shape(self):
        return (self.shape[0], self.shape[2])

    y_shape = output_shape

    def pack(self, codes, stream=None):
        """The codes laid out for the kernel, in a new uint8 tensor.  It belongs
        to `stream`, like any tensor that torch makes there: another stream waits
        for that one before it reads it."""
        import torch
        _, c_in, c_out = self.shape
        dev = self._on_device()
        pc = _check("codes", codes, (c_out, (c_in + 1) // 2), self._u8, dev)
        with _allocating_on(stream, codes.device):
            packed = torch.empty(self.packed_bytes, dtype=torch.uint8, device=codes.device)
        rc = self._lib.conv_w4_pack(c_in, c_out, pc, packed.data_ptr(), _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_w4_pack", rc)
        return packed

    def run(self, x, packed, scales, bias, y, stream=None) -> None:  # noqa: D401
        """Enqueue the layer on `stream` (default: torch's current stream)."""
        sx, sw, ss, sb, sy = self._shapes
        dt, dev = self._dt, self._on_device()
        px, pw, ps = _check("x", x, sx, dt, dev), _check("packed", packed, sw, self._u8, dev), _check("scales", scales, ss, dt, dev)
        pb = None if bias is None else _check("bias", bias, sb, self._f32, dev)
        py = _check("y", y, sy, dt, dev)
        rc = self._lib.conv_run_w4(self._handle, px, pw, ps, pb, py, _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_run_w4", rc)


_BLOCKNORM_MAPS = {"x", "f", "y", "z", "dy", "dz", "dx", "df"}
_BLOCKNORM_RUN = ("x", "f", "y", "z", "stats", "scale", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta")
_BLOCKNORM_BWD = ("x", "f", "dy", "dz", "dx", "df", "stats", "scale", "gate", "post_gamma", "post_beta", "pre_gamma",
                  "dscale", "dgate", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")


class BlockNormPlan(_MapPlan):
    """The norms before and after a block, fused with the block's gate, its
    residual scale and the residual add (conv_plan_create_blocknorm)::

        y = x + scale * gate * (post(f) * post_gamma + post_beta)
        z = pre(y) * pre_gamma + pre_beta

    x is the residual stream and f the block's output; ``post`` and ``pre`` are
    "layer", "rms" or "none", over each pixel's channels.  Maps (x, f, y, z and
    their gradients) are [n, h, w, c] CUDA tensors, dense or channel slices of a
    wider dense buffer; gate and dgate float32 [n, c], the other parameters and
    their gradients float32 [c]; stats float32 [n, h, w, 4].  A parameter that is
    None is 1 (scale, gate, gammas) or 0 (betas)."""

    def __init__(self, n, h, w, c, post="layer", pre="layer", eps=1e-5, dtype="bf16"):
        self.shape = (n, h, w, c)
        self.post, self.pre, self.eps, self.dtype, self.act = post, pre, eps, dtype, "none"
        self._create("conv_plan_create_blocknorm", n, h, w, c, NORMS[post], NORMS[pre], float(eps), DTYPES[dtype])
        self._cshape, self._gshape, self._sshape = (c,), (n, c), (n, h, w, 4)
        self._known = {}  # shapes and types of a call's tensors, by which of them are given

    @property
    def output_shape(self):
        return self.shape

    y_shape = output_shape

    def _addresses(self, names, tensors):
        """Addresses of a call's tensors (None where there is none) and the pixel
        pitches of its maps (0: dense).  Maps come first in `names`."""
        none = tuple([t is None for t in tensors])
        known = self._known.get(none)  # (as long as the call's tensors: forward and gradient differ)
        if known is None:
            maps = [k for k in names if k in _BLOCKNORM_MAPS]
            shape = {"stats": self._sshape, "gate": self._gshape, "dgate": self._gshape, **{k: self.shape for k in maps}}
            given = [k for k, absent in zip(names, none) if not absent]
            known = (given, [shape.get(k, self._cshape) for k in given],
                     [self._dt if k in maps else self._f32 for k in given], [self._device] * len(given), len(maps))
            self._known[none] = known
        given, shapes, dtypes, devices, maps = known
        ts = tensors if len(given) == len(names) else [t for t in tensors if t is not None]
        pitches = [0] * maps
        shape_of, dtype_of, dense, device_of, address, _ = _tensor_getters()
        try:
            good = list(map(shape_of, ts)) == shapes and list(map(dtype_of, ts)) == dtypes and list(map(device_of, ts)) == devices
            whole = list(map(dense, ts))
            if good and False in whole:  # slices, unless it is no map
                for k, t, flat in zip(given, ts, whole):
                    if not flat and k in _BLOCKNORM_MAPS:
                        pitches[names.index(k)] = self._pitch(k, t)
                    good = good and (flat or k in _BLOCKNORM_MAPS)
            found = list(map(address, ts))
        except (AttributeError, TypeError):  # (not tensors)
            good = False
        if not good:  # what is to be refused: one by one
            found = []
            for k, t, shape, dtype in zip(given, ts, shapes, dtypes):
                if k in _BLOCKNORM_MAPS:
                    at, pitches[names.index(k)] = self._map(k, t)
                    found.append(at)
                else:
                    found.append(_check(k, t, shape, dtype, self._device))
        if len(given) != len(names):
            it = iter(found)
            found = [None if absent else next(it) for absent in none]
        return found, pitches

    def run(self, x, f, y, z, stats=None, scale=None, gate=None, post_gamma=None, post_beta=None, pre_gamma=None,
            pre_beta=None, stream=None) -> None:  # noqa: D401
        """Enqueue y and z on `stream` (default: torch's current stream).

        f None (``post`` "none"): z is the norm of x, and y is None.  y may be
        None where there is a z; z is None where ``pre`` is "none".  y or z may
        be x or f itself.  stats, where given, is what the gradient needs."""
        dev = self._on_device()
        if x is None:
            raise ValueError("x is missing")
        p, (ix, jf, iy, iz) = self._addresses(_BLOCKNORM_RUN, (x, f, y, z, stats, scale, gate, post_gamma, post_beta,
                                                               pre_gamma, pre_beta))
        rc = self._lib.conv_run_blocknorm(self._handle, p[0], ix, p[1], jf, _BlockNormPointers(*p[5:]), p[2], iy, p[3], iz,
                                          p[4], _stream_handle(stream, dev))
        if rc != 0:
            raise ConvError("conv_run_blocknorm", rc)

    def run_backward(self, x, f, stats, dy, dz, dx, df, scale=None, gate=None, post_gamma=None, post_beta=None,
                     pre_gamma=None, dscale=None, dgate=None, dpost_gamma=None, dpost_beta=None, dpre_gamma=None,
                     dpre_beta=None, stream=None) -> None:
        """Enqueue the gradient: dx and df, and those of the parameters where
        given.  x, f, stats and the parameters as the forward run had them; dy
        None is 0; dx or df may be any of the maps that are read."""
        dev = self._on_device()
        if x is None or stats is None or dx is None:
            raise ValueError("x, stats or dx is missing")
        p, (ix, jf, iy, iz, kx, kf) = self._addresses(
            _BLOCKNORM_BWD, (x, f, dy, dz, dx, df, stats, scale, gate, post_gamma, post_beta, pre_gamma, dscale, dgate,
                             dpost_gamma, dpost_beta, dpre_gamma, dpre_beta))
        handle = _stream_handle(stream, dev)
        take, give = _raw_memory_calls()
        ws = take(self.workspace_bytes_backward, handle) if self.workspace_bytes_backward else None
        try:
            rc = self._lib.conv_run_blocknorm_bwd(self._handle, p[0], ix, p[1], jf, _BlockNormPointers(*p[7:12]), p[6], p[2],
                                                  iy, p[3], iz, p[4], kx, p[5], kf, _BlockNormPointers(*p[12:]), ws, handle)
        finally:
            if ws is not None:
                give(ws)
        if rc != 0:
            raise ConvError("conv_run_blocknorm_bwd", rc)


class GradClipPlan(_OpPlan):
    """The global norm of many gradients, and clipping (conv_plan_create_gradclip)::

        norm = sqrt(sum of all squares)
        out = min(1, max_norm / (norm + 1e-6)) * g

    ``shapes``: a shape (or a number of elements) for each tensor, of which the
    number of elements counts; ``dtypes``: "bf16" or "f32" for all of them, or
    one for each."""

    def __init__(self, shapes, dtypes="bf16"):
        import math
        self.shapes = [(s,) if isinstance(s, int) else tuple(s) for s in shapes]
        count = len(self.shapes)
        names = [dtypes] * count if isinstance(dtypes, str) else list(dtypes)
        if len(names) != count:
            raise ValueError(f"{len(names)} dtypes for {count} tensors")
        self.dtypes, self.act = names, "none"
        self.dtype, self.shape = (names[0] if names else "f32"), (count,)
        self._counts = [math.prod(s) for s in self.shapes]
        counts = (ctypes.c_int64 * count)(*self._counts)
        codes = (ctypes.c_int * count)(*(DTYPES[d] for d in names))
        self._create("conv_plan_create_gradclip", count, counts, codes)
        self._dtypes, self._devices = [_torch_dtype(d) for d in names], [self._device] * count

    @property
    def output_shape(self):
        return ()

    y_shape = output_shape

    def _addresses(self, name, tensors):
        """The tensors' addresses, one after the other in memory of the host."""
        if len(tensors) != len(self._counts):
            raise ValueError(f"{len(tensors)} {name} for a plan of {len(self._counts)}")
        _, dtype_of, dense, device_of, address, count_of = _tensor_getters()
        try:
            if (list(map(dtype_of, tensors)) == self._dtypes and list(map(device_of, tensors)) == self._devices and
                    list(map(count_of, tensors)) == self._counts and all(map(dense, tensors))):
                return array("Q", map(address, tensors))
        except (AttributeError, TypeError):  # (not tensors)
            pass
        return array("Q", [_check(f"{name}[{i}]", t, t.shape if t is not None and t.numel() == k else self.shapes[i], d, self._device)
                           for i, (t, k, d) in enumerate(zip(tensors, self._counts, self._dtypes))])

    def run(self, grads, max_norm, norm, out=None, stream=None) -> None:  # noqa: D401
        """Enqueue the norm (a float32 scalar tensor) and the clipped gradients
        on `stream` (default: torch's current stream): into the tensors of `out`
        (any of which may be the gradient itself), or in place.  max_norm
        infinite: the norm alone.  A norm that is not finite (or passes the
        largest float32 number) clips nothing: leave that step out."""
        dev = self._on_device()
        g = self._addresses("grads", grads)
        o = None if out is None else self._addresses("out", out)
        pn = _check("norm", norm, (), self._f32, dev)
        handle = _stream_handle(stream, dev)
        take, give = _raw_memory_calls()
        ws = take(self.workspace_bytes, handle) if self.workspace_bytes else None
        try:
            rc = self._lib.conv_run_gradclip(self._handle, g.buffer_info()[0], None if o is None else o.buffer_info()[0],
                                             float(max_norm), pn, ws, handle)
        finally:
            if ws is not None:
                give(ws)
        if rc != 0:
            raise ConvError("conv_run_gradclip", rc)


def w4_quantize(w, group=128, stream=None):
    """Codes and scales of float weights [c_out, c_in] (conv_w4_quantize), new
    tensors that belong to `stream` as W4Plan.pack's does."""
    import torch
    dt = _dtype_name(w)
    if len(w.shape) != 2 or group < 1:
        raise ValueError(f"w must be [c_out, c_in] and group positive, got {tuple(w.shape)} and {group}")
    c_out, c_in = w.shape
    dev = _current_device()
    pw = _check("w", w, (c_out, c_in), w.dtype, dev)
    with _allocating_on(stream, w.device):
        codes = torch.empty(c_out, (c_in + 1) // 2, dtype=torch.uint8, device=w.device)
        scales = torch.empty(c_out, -(-c_in // group), dtype=w.dtype, device=w.device)
    rc = load_library().conv_w4_quantize(c_in, c_out, group, DTYPES[dt], pw, codes.data_ptr(), scales.data_ptr(),
                                         _stream_handle(stream, dev))
    if rc != 0:
        raise ConvError("conv_w4_quantize", rc)
    return codes, scales
