"""Python binding of libsdpa (argument marshalling only).

Every computation happens in the CUDA kernels of ``libsdpa.so``; this module
only checks tensor metadata, passes device pointers, sizes and the current
CUDA stream to the C ABI declared in ``include/sdpa.h``, and turns a status
code into an exception.  There is no CPU or PyTorch fallback: if the library
or a CUDA device is missing, calls raise.

    import scaled_dot_product_13_b200 as sdpa
    out = sdpa.forward(q, k, v, scale=None, causal=True, window_size=0)
    dq, dk, dv = sdpa.backward(q, k, v, out, lse, dout, causal=True)   # lse from forward_ex
    q, k = sdpa.rotary(sdpa.rotary_plan(128), q, k)

q [B, Hq, L, Dqk], k [B, Hkv, S, Dqk], v [B, Hkv, S, Dv], contiguous CUDA
tensors of one dtype (bfloat16 or float16).  Query head hq reads KV head
hq // (Hq // Hkv); query i sits at key position i + S - L.

No call records anything for autograd: results carry no graph, also where inputs
require grad (use ``backward`` and ``rotary(..., inverse=True)`` in a
``torch.autograd.Function``).

``stream`` (a torch stream or a handle; default the current one): where a call
runs.  Tensors that a call makes are that stream's, as under
``torch.cuda.stream(stream)``, and may be used on the stream that is current at the
call once that waits for it; what a call is given must be ready on ``stream``.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = ["forward", "forward_ws", "forward_noalloc", "forward_ex", "Options", "workspace_bytes", "plan", "device_status",
           "backward", "backward_workspace_bytes", "BackwardOptions",
           "rotary", "rotary_plan", "RotaryPlan", "ROPE_SCALINGS",
           "set_wait_limit_ns", "watchdog_selftest", "exp2_selftest", "time_next_main_kernel", "time_next_call", "load_library", "library_path",
           "SdpaError", "PATH_AUTO", "PATH_SPLITKV", "PATH_TC", "PATH_TC2", "PATH_WIDE", "PATH_TC_DUAL", "PATH_TC_KSPLIT",
           "PATH_TC2_LOOP", "STATUS"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB: ctypes.CDLL | None = None

PATH_AUTO, PATH_SPLITKV, PATH_TC, PATH_TC2, PATH_WIDE, PATH_TC_DUAL, PATH_TC_KSPLIT, PATH_TC2_LOOP = \
    0, 1, 2, 3, 4, 5, 6, 7
STATUS = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID_ARG", 2: "SDPA_ERR_UNSUPPORTED",
          3: "SDPA_ERR_RESOURCES", 4: "SDPA_ERR_CUDA", 5: "SDPA_ERR_TIMEOUT"}


class SdpaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class Options(ctypes.Structure):
    """Mirror of sdpa_options."""
    _fields_ = [("has_q_offset", ctypes.c_int), ("q_offset", ctypes.c_int),
                ("sinks", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("force_path", ctypes.c_int), ("force_splits", ctypes.c_int)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("splits", ctypes.c_int), ("rows", ctypes.c_int),
                ("row_tile", ctypes.c_int), ("row_tiles", ctypes.c_int),
                ("key_block", ctypes.c_int), ("keys_per_split", ctypes.c_int),
                ("ctas", ctypes.c_int), ("launches", ctypes.c_int), ("dqk_pad", ctypes.c_int),
                ("dv_pad", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class BackwardOptions(ctypes.Structure):
    """Mirror of sdpa_backward_options."""
    _fields_ = [("has_q_offset", ctypes.c_int), ("q_offset", ctypes.c_int),
                ("sinks", ctypes.c_void_p), ("dsinks", ctypes.c_void_p), ("dlse", ctypes.c_void_p),
                ("weight_terms", ctypes.c_int)]


class RotaryConfig(ctypes.Structure):
    """Mirror of sdpa_rotary_config."""
    _fields_ = [("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("base", ctypes.c_double), ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_int), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("magnitude", ctypes.c_double)]


class RotaryPlan(ctypes.Structure):
    """Mirror of sdpa_rotary_plan: host memory only, filled by ``rotary_plan``."""
    _fields_ = [("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("magnitude", ctypes.c_float), ("turns", ctypes.c_uint64 * 256)]


class Strides(ctypes.Structure):
    """Mirror of sdpa_strides."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("token", ctypes.c_longlong)]


class RotaryTensor(ctypes.Structure):
    """Mirror of sdpa_rotary_tensor."""
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("x_strides", Strides), ("out_strides", Strides)]


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}


def library_path() -> str:
    return os.environ.get("SDPA_LIBRARY", os.path.join(_HERE, "libsdpa.so"))


def load_library() -> ctypes.CDLL:
    """Load libsdpa.so (raises if it was not built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libsdpa.so not found at {path}; build it with "
                           "`python -m scaled_dot_product_13_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    common = [vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, i]
    lib.sdpa_forward.argtypes = common + [vp]
    lib.sdpa_forward_ws.argtypes = common + [vp, sz, vp]
    lib.sdpa_forward_noalloc.argtypes = common + [vp]
    lib.sdpa_forward_ex.argtypes = common + [ctypes.POINTER(Options), vp, sz, vp]
    lib.sdpa_forward_planned.argtypes = common + [i, i, vp, sz, vp]
    lib.sdpa_workspace_bytes.argtypes = [i] * 10
    lib.sdpa_workspace_bytes.restype = sz
    lib.sdpa_plan.argtypes = [i] * 13 + [ctypes.POINTER(PlanInfo)]
    lib.sdpa_backward.argtypes = [vp] * 9 + [i] * 7 + [f, i, i, i, ctypes.POINTER(BackwardOptions), vp, sz, vp]
    lib.sdpa_backward_workspace_bytes.argtypes = [i] * 10 + [ctypes.POINTER(BackwardOptions)]
    lib.sdpa_backward_workspace_bytes.restype = sz
    ll = ctypes.c_longlong
    lib.sdpa_rotary_init.argtypes = [ctypes.POINTER(RotaryConfig), ctypes.POINTER(RotaryPlan)]
    lib.sdpa_rotary.argtypes = [ctypes.POINTER(RotaryPlan), vp, i, i, i, vp, i, ll, ll,
                                i, i, vp]
    lib.sdpa_device_status.argtypes = [i]
    lib.sdpa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.sdpa_set_wait_limit_ns.restype = None
    lib.sdpa_watchdog_selftest.argtypes = [ctypes.c_uint64, ctypes.POINTER(ctypes.c_int)]
    lib.sdpa_exp2_selftest.argtypes = [ctypes.c_float, ctypes.c_float, i, vp, vp]
    lib.sdpa_time_next_main_kernel.argtypes = [vp, vp]
    lib.sdpa_time_next_main_kernel.restype = None
    lib.sdpa_time_next_call.argtypes = [vp, vp, vp]
    lib.sdpa_time_next_call.restype = None
    lib.sdpa_status_string.restype = ctypes.c_char_p
    lib.sdpa_status_string.argtypes = [i]
    lib.sdpa_last_error_message.restype = ctypes.c_char_p
    for fn in ("sdpa_forward", "sdpa_forward_ws", "sdpa_forward_noalloc", "sdpa_forward_ex",
               "sdpa_forward_planned", "sdpa_plan", "sdpa_rotary_init", "sdpa_rotary", "sdpa_backward",
               "sdpa_device_status", "sdpa_watchdog_selftest", "sdpa_exp2_selftest"):
        getattr(lib, fn).restype = ctypes.c_int
    _LIB = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        msg = load_library().sdpa_last_error_message().decode(errors="replace")
        raise SdpaError(status, msg)


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise SdpaError(2, f"dtype {t.dtype} is not supported (bfloat16 or float16)")


def _shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise SdpaError(1, "q, k, v must be 4-D [B, H, N, D]")
    B, Hq, L, Dqk = q.shape
    Bk, Hkv, S, Dk = k.shape
    Bv, Hv, Sv, Dv = v.shape
    if (Bk, Dk) != (B, Dqk) or (Bv, Hv, Sv) != (B, Hkv, S):
        raise SdpaError(1, f"inconsistent shapes q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise SdpaError(1, f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise SdpaError(1, f"{name} must be contiguous")
        if t.dtype != q.dtype:
            raise SdpaError(1, "q, k, v must share one dtype")
    return int(B), int(Hq), int(Hkv), int(L), int(S), int(Dqk), int(Dv)


def _stream(stream):
    import torch

    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on ``stream`` (None: the current one) to write.  Its
    memory is that stream's, so that nothing pending on another stream still uses it;
    and as the current stream is where it is likely read, it is not given to a later
    call before the work that is on the current stream when it is released is done."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    if here != stream:
        t.record_stream(here)
    return t


def _out_like(q, L, Dv, out, stream):
    B, Hq = q.shape[0], q.shape[1]
    if out is None:
        return _empty((B, Hq, L, Dv), q.dtype, q.device, stream)
    if tuple(out.shape) != (B, Hq, L, Dv) or out.dtype != q.dtype or not out.is_contiguous():
        raise SdpaError(1, "out must be a contiguous [B, Hq, L, Dv] tensor of q's dtype")
    return out


def forward(q, k, v, scale: float | None = None, causal: bool = False, window_size: int = 0,
            out=None, stream=None):
    """Fused attention forward; returns out [B, Hq, L, Dv] (same dtype as q)."""
    lib = load_library()
    B, Hq, Hkv, L, S, Dqk, Dv = _shapes(q, k, v)
    sc = float(Dqk ** -0.5 if scale is None else scale)
    out = _out_like(q, L, Dv, out, stream)
    _check(lib.sdpa_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq,
                            Hkv, L, S, Dqk, Dv, sc, int(bool(causal)), int(window_size),
                            _dtype_code(q), _stream(stream)))
    return out


def forward_noalloc(q, k, v, scale: float | None = None, causal: bool = False,
                    window_size: int = 0, out=None, stream=None):
    """As ``forward``, through sdpa_forward_noalloc: no device allocation in
    the library; split partials go to the library's fixed 16 MiB per-device
    scratch array.  ``out`` should be preallocated by callers that cannot
    allocate (when None, this wrapper allocates it with torch).  Calls that
    overlap on the GPU share that array and race; keep them on one stream."""
    lib = load_library()
    B, Hq, Hkv, L, S, Dqk, Dv = _shapes(q, k, v)
    sc = float(Dqk ** -0.5 if scale is None else scale)
    out = _out_like(q, L, Dv, out, stream)
    _check(lib.sdpa_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B,
                                    Hq, Hkv, L, S, Dqk, Dv, sc, int(bool(causal)),
                                    int(window_size), _dtype_code(q), _stream(stream)))
    return out


def forward_ex(q, k, v, scale: float | None = None, causal: bool = False, window_size: int = 0,
               q_offset: int | None = None, sinks=None, lse=None, out=None, stream=None,
               workspace=None, force_path: int = 0, force_splits: int = 0):
    """sdpa_forward_ex: ``q_offset`` = key position of query row 0 (default
    S - L); ``sinks`` = optional float32 CUDA tensor [Hq] of sink logits;
    ``lse`` = optional float32 CUDA tensor [B, Hq, L] that receives each row's
    log-sum-exp.  ``workspace``: as ``forward_ws`` (None = pool allocation)."""
    import torch

    lib = load_library()
    B, Hq, Hkv, L, S, Dqk, Dv = _shapes(q, k, v)
    sc = float(Dqk ** -0.5 if scale is None else scale)
    out = _out_like(q, L, Dv, out, stream)
    opt = Options()
    if q_offset is not None:
        opt.has_q_offset, opt.q_offset = 1, int(q_offset)
    for name, t, shape in (("sinks", sinks, (Hq,)), ("lse", lse, (B, Hq, L))):
        if t is None:
            continue
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
                and tuple(t.shape) == shape):
            raise SdpaError(1, f"{name} must be a contiguous float32 CUDA tensor of shape {shape}")
    opt.sinks = sinks.data_ptr() if sinks is not None else None
    opt.lse = lse.data_ptr() if lse is not None else None
    opt.force_path, opt.force_splits = int(force_path), int(force_splits)
    ws_ptr = 0 if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.sdpa_forward_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq,
                               Hkv, L, S, Dqk, Dv, sc, int(bool(causal)), int(window_size),
                               _dtype_code(q), ctypes.byref(opt), ws_ptr, ws_bytes,
                               _stream(stream)))
    return out


def forward_ws(q, k, v, workspace, scale: float | None = None, causal: bool = False,
               window_size: int = 0, out=None, stream=None, force_path: int = 0,
               force_splits: int = 0):
    """As ``forward`` with a caller-owned workspace tensor (any dtype, on the
    device, at least ``workspace_bytes`` bytes; may be None when that is 0).
    ``force_path`` / ``force_splits`` pin the router (0 = its choice)."""
    lib = load_library()
    B, Hq, Hkv, L, S, Dqk, Dv = _shapes(q, k, v)
    sc = float(Dqk ** -0.5 if scale is None else scale)
    out = _out_like(q, L, Dv, out, stream)
    ws_ptr = 0 if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.sdpa_forward_planned(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    B, Hq, Hkv, L, S, Dqk, Dv, sc, int(bool(causal)),
                                    int(window_size), _dtype_code(q), int(force_path),
                                    int(force_splits), ws_ptr, ws_bytes, _stream(stream)))
    return out


def workspace_bytes(B, Hq, Hkv, L, S, Dqk, Dv, causal=False, window_size=0, dtype="bf16",
                    force_path: int = 0, force_splits: int = 0, num_sms: int | None = None) -> int:
    """Workspace a call needs (router's plan, or the pinned one)."""
    return plan(B, Hq, Hkv, L, S, Dqk, Dv, causal, window_size, dtype, num_sms=num_sms,
                force_path=force_path, force_splits=force_splits)["workspace_bytes"]


def plan(B, Hq, Hkv, L, S, Dqk, Dv, causal=False, window_size=0, dtype="bf16",
         num_sms: int | None = None, force_path: int = 0, force_splits: int = 0) -> dict:
    """The router's decision for one problem (host only)."""
    lib = load_library()
    if num_sms is None:
        num_sms = _num_sms()
    info = PlanInfo()
    dt = 0 if dtype in ("bf16", "bfloat16") else 1
    _check(lib.sdpa_plan(B, Hq, Hkv, L, S, Dqk, Dv, int(bool(causal)), int(window_size), dt,
                         int(num_sms), int(force_path), int(force_splits), ctypes.byref(info)))
    return info.as_dict()


def backward_workspace_bytes(B, Hq, Hkv, L, S, Dqk, Dv, causal=False, window_size=0, dtype="bf16",
                             q_offset: int | None = None, weight_terms: int = 0) -> int:
    """Workspace that ``backward`` needs for this problem on the current device."""
    lib = load_library()
    opt = BackwardOptions()
    if q_offset is not None:
        opt.has_q_offset, opt.q_offset = 1, int(q_offset)
    opt.weight_terms = int(weight_terms)
    n = lib.sdpa_backward_workspace_bytes(B, Hq, Hkv, L, S, Dqk, Dv, int(bool(causal)), int(window_size),
                                          0 if dtype in ("bf16", "bfloat16") else 1, ctypes.byref(opt))
    if n == 0:
        msg = lib.sdpa_last_error_message().decode(errors="replace")
        raise SdpaError(1, msg)
    return n


def backward(q, k, v, out, lse, dout, scale: float | None = None, causal: bool = False, window_size: int = 0,
             q_offset: int | None = None, sinks=None, dlse=None, dq=None, dk=None, dv=None, dsinks=None,
             stream=None, workspace=None, weight_terms: int = 0):
    """Gradients (dq, dk, dv) of ``forward_ex(q, k, v, ..., lse=lse)``, given its
    ``out`` and ``lse`` and the gradient ``dout`` of out; the other arguments as
    in that call.  ``dlse``: gradient [B, Hq, L] (float32) of lse, where it was
    used.  ``dsinks``: float32 [Hq] that receives the gradient of ``sinks``.
    ``dq`` / ``dk`` / ``dv``: contiguous tensors to write (new ones when None).
    ``weight_terms``: 16-bit terms that P and dS enter their products as, 1 or 2: the
    gradients' error is up to 1.45 times that of exact weights with 1, not noticeably
    above it with 2, which takes up to 1.4 times as long (0: 2 up to B Hq L S = 2^20,
    where it costs 0 to 30 %).
    Rows with lse = -inf take no part (their q and dout must be finite).  Out and lse
    merged over chunks of keys: add up the calls' dq, but take dsinks from one.
    ``workspace``: at least ``backward_workspace_bytes`` bytes on the device,
    not used by other work until the call's kernels are done.  None: from
    torch's caching allocator on the current stream, or, with ``stream`` given,
    from the stream-ordered pool."""
    import torch

    lib = _LIB or load_library()
    dtype, device, f32 = q.dtype, q.device, torch.float32
    qs, ks, vs = q.shape, k.shape, v.shape
    if not (len(qs) == len(ks) == 4 and vs[:-1] == ks[:-1] and ks[0] == qs[0] and ks[3] == qs[3]
            and q.is_cuda and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
            and k.dtype == dtype and v.dtype == dtype):
        _shapes(q, k, v)  # names what is wrong
    if k.device != device or v.device != device:
        raise SdpaError(1, "k and v must be on q's device")
    dt = _dtype_code(q)
    B, Hq, L, Dqk = qs
    Hkv, S, Dv = ks[1], ks[2], vs[3]
    rows = (B, Hq, L)

    def want(name, t, shape, kind):
        if t.shape != shape or t.dtype != kind or t.device != device or not t.is_contiguous():
            raise SdpaError(1, f"{name} must be a contiguous {kind} tensor of shape {tuple(shape)} on q's device")
        return t.data_ptr()

    if out is None or lse is None or dout is None:
        raise SdpaError(1, "out, lse and dout are needed")
    opt = BackwardOptions()
    if q_offset is not None:
        opt.has_q_offset, opt.q_offset = 1, int(q_offset)
    if sinks is not None:
        opt.sinks = want("sinks", sinks, (Hq,), f32)
    if dsinks is not None:
        opt.dsinks = want("dsinks", dsinks, (Hq,), f32)
    if dlse is not None:
        opt.dlse = want("dlse", dlse, rows, f32)
    if weight_terms:
        opt.weight_terms = int(weight_terms)
    opt = ctypes.byref(opt)
    causal, window_size = 1 if causal else 0, int(window_size)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return backward(q, k, v, out, lse, dout, scale, causal, window_size, q_offset, sinks, dlse, dq, dk, dv,
                            dsinks, stream, workspace, weight_terms)
    if stream is None:  # (q, k and v are contiguous)
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
    else:
        dq = _empty(qs, dtype, device, stream) if dq is None else dq
        dk = _empty(ks, dtype, device, stream) if dk is None else dk
        dv = _empty(vs, dtype, device, stream) if dv is None else dv
    ws_ptr = ws_bytes = 0
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise SdpaError(1, "workspace must be contiguous and on q's device")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif stream is None:
        ws_bytes = lib.sdpa_backward_workspace_bytes(B, Hq, Hkv, L, S, Dqk, Dv, causal, window_size, dt, opt)
        if ws_bytes:  # (invalid problems are left for the call to name)
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
            ws_ptr = workspace.data_ptr()
    st = lib.sdpa_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), want("out", out, rows + (Dv,), dtype),
                           want("lse", lse, rows, f32), want("dout", dout, rows + (Dv,), dtype),
                           want("dq", dq, qs, dtype), want("dk", dk, ks, dtype),
                           want("dv", dv, vs, dtype), B, Hq, Hkv, L, S, Dqk, Dv,
                           Dqk ** -0.5 if scale is None else scale, causal, window_size, dt, opt, ws_ptr, ws_bytes,
                           _call_stream(stream, device))
    if st:
        _check(st)
    return dq, dk, dv


def rotary_plan(head_dim: int, rotary_dim: int | None = None, base: float = 10000.0,
                interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                original_length: int = 0, beta_fast: float | None = None,
                beta_slow: float | None = None, magnitude: float | None = None) -> RotaryPlan:
    """The frequencies of ``rotary``, computed once on the host (no CUDA call).
    ``scaling``: "none", "linear", "ntk", "yarn" or "banded", with ``factor``
    and (yarn, banded) ``original_length``; see sdpa_rotary_config."""
    if scaling not in ROPE_SCALINGS:
        raise SdpaError(1, f"scaling must be one of {', '.join(ROPE_SCALINGS)} (got {scaling!r})")
    for name, x in (("rotary_dim", rotary_dim), ("base", base), ("beta_fast", beta_fast),
                    ("beta_slow", beta_slow), ("magnitude", magnitude)):
        if x is not None and x == 0:  # 0 means "default" in the C structure
            raise SdpaError(1, f"{name} must not be 0")
    cfg = RotaryConfig(int(head_dim), int(rotary_dim or 0), int(bool(interleaved)), float(base),
                       ROPE_SCALINGS[scaling], float(factor), int(original_length),
                       float(beta_fast or 0), float(beta_slow or 0), float(magnitude or 0))
    out = RotaryPlan()
    _check(load_library().sdpa_rotary_init(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def _call_stream(stream, device):
    """The handle of ``stream``, by default the current stream of ``device``."""
    import torch

    if stream is None:
        # without the Stream object that current_stream makes: 0.2 us, not 2.4; but the
        # function is torch's own and may be gone from another version
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def rotary(plan: RotaryPlan, q, k=None, positions=None, offset: int = 0, inverse: bool = False,
           out_q=None, out_k=None, stream=None):
    """Rotate ``q`` (and ``k``) [B, H, L, head_dim] by their positions; returns
    the result(s).  Any strides with a contiguous last dim: a projection
    [B, L, H, D] goes in as ``x.transpose(1, 2)``.  ``positions``: int32 or
    int64 CUDA tensor [L], [1, L] or [B, L] (default 0..L-1), ``offset`` added.
    ``inverse=True`` is the gradient.  ``out_q`` / ``out_k``: views to write
    (the inputs themselves: in place); by default new dense [B, H, L, D]."""
    import torch

    lib = _LIB or load_library()
    if not isinstance(plan, RotaryPlan):
        raise SdpaError(1, "plan must come from rotary_plan")
    if k is None and out_k is not None:
        raise SdpaError(1, "out_k without k")
    if q.dim() != 4 or not q.is_cuda:
        raise SdpaError(1, f"q must be a CUDA tensor [B, H, L, {plan.head_dim}]")
    B, Hq, L, D = q.shape
    dtype, device = q.dtype, q.device
    dt = _dtype_code(q)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return rotary(plan, q, k, positions, offset, inverse, out_q, out_k, stream)
    out_q, fields = _rotary_tensor("q", q, out_q, plan.head_dim, B, L, dtype, device, stream)
    if k is not None:
        out_k, more = _rotary_tensor("k", k, out_k, plan.head_dim, B, L, dtype, device, stream)
        fields += more
    pos_ptr, bits, pos_stride = None, 0, 0
    if positions is not None:
        if positions.device != device or positions.dtype not in (torch.int32, torch.int64):
            raise SdpaError(1, "positions must be an int32 or int64 tensor on q's device")
        shape = positions.shape
        if not (len(shape) in (1, 2) and shape[-1] == L and (len(shape) == 1 or shape[0] in (1, B))) \
                or (L > 1 and positions.stride(-1) != 1):
            raise SdpaError(1, f"positions must be [L], [1, L] or [B, L] with L = {L}, contiguous along L")
        pos_ptr, bits = positions.data_ptr(), 32 if positions.dtype == torch.int32 else 64
        if len(shape) == 2 and shape[0] == B and B > 1:
            pos_stride = positions.stride(0)
    count = len(fields) // 9
    st = lib.sdpa_rotary(plan, struct.pack(_ROTARY_TENSOR * count, *fields), count, B, L, pos_ptr, bits, pos_stride,
                         offset, 1 if inverse else 0, dt, _call_stream(stream, device))
    if st:
        _check(st)
    return out_q if k is None else (out_q, out_k)


# sdpa_rotary_tensor: x, out, heads, x's strides, out's strides
_ROTARY_TENSOR = "QQi4xqqqqqq"


def _rotary_tensor(name, x, out, D, B, L, dtype, device, stream):
    """The checked output of one tensor, and the fields of its sdpa_rotary_tensor."""
    shape = x.shape
    if len(shape) != 4 or shape[3] != D:
        raise SdpaError(1, f"{name} must be [B, H, L, {D}] (got {tuple(shape)})")
    if x.device != device or x.dtype != dtype or shape[0] != B or shape[2] != L:
        raise SdpaError(1, "q and k must share device, dtype, batch and length")
    xb, xh, xt, xd = x.stride()
    if xd != 1:
        raise SdpaError(1, f"{name}'s last dim must be contiguous")
    if out is None:
        out = _empty(shape, dtype, device, stream)
    elif out.shape != shape or out.dtype != dtype or out.device != device or out.stride(3) != 1:
        raise SdpaError(1, f"out_{name} must have {name}'s shape, dtype and device, its last dim contiguous")
    ob, oh, ot, _ = out.stride()
    return out, (x.data_ptr(), out.data_ptr(), shape[1], xb, xh, xt, ob, oh, ot)


def _num_sms() -> int:
    try:
        import torch

        if torch.cuda.is_available():
            return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    except Exception:  # pragma: no cover
        pass
    return 148


def device_status(clear: bool = True) -> None:
    """Synchronise and raise SdpaError(SDPA_ERR_TIMEOUT) if a kernel's bounded
    wait expired since the last clear."""
    _check(load_library().sdpa_device_status(int(bool(clear))))


def time_next_main_kernel(start_event, stop_event) -> None:
    """Arm the profiling hook: the next call on this thread records the two
    torch.cuda.Event objects around its main attention kernel.  The events
    must already hold a CUDA handle (record them once beforehand)."""
    if not start_event.cuda_event or not stop_event.cuda_event:
        raise SdpaError(1, "events have no CUDA handle yet; record them once first")
    load_library().sdpa_time_next_main_kernel(ctypes.c_void_p(start_event.cuda_event),
                                              ctypes.c_void_p(stop_event.cuda_event))


def time_next_call(start_event, stop_event, call_event) -> None:
    """As ``time_next_main_kernel``, plus ``call_event`` recorded after the
    call's last launch (the combine, when the keys are split).  Any of the
    three may be None (not recorded)."""
    handles = []
    for e in (start_event, stop_event, call_event):
        if e is not None and not e.cuda_event:
            raise SdpaError(1, "events have no CUDA handle yet; record them once first")
        handles.append(ctypes.c_void_p(e.cuda_event if e is not None else None))
    load_library().sdpa_time_next_call(*handles)


def exp2_selftest(lo: float, hi: float, n: int, device="cuda"):
    """(poly, ref): the kernels' FMA-pipe exp2 and exp2f on n points over
    [lo, hi], as fp32 CUDA tensors."""
    import torch

    poly = torch.empty(n, dtype=torch.float32, device=device)
    ref = torch.empty(n, dtype=torch.float32, device=device)
    _check(load_library().sdpa_exp2_selftest(ctypes.c_float(lo), ctypes.c_float(hi), int(n),
                                             ctypes.c_void_p(poly.data_ptr()),
                                             ctypes.c_void_p(ref.data_ptr())))
    torch.cuda.synchronize()
    return poly, ref


def set_wait_limit_ns(ns: int) -> None:
    load_library().sdpa_set_wait_limit_ns(int(ns))


def watchdog_selftest(limit_ns: int = 100_000_000) -> int:
    """Run the watchdog self-test kernel; returns 0 when its wait expired."""
    res = ctypes.c_int(-1)
    _check(load_library().sdpa_watchdog_selftest(int(limit_ns), ctypes.byref(res)))
    return res.value
