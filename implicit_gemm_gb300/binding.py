"""ctypes binding of libwgrad.so (include/wgrad.h).  Argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors may be
torch tensors (their data_ptr() is passed) or plain integer device addresses.
The library must have been built (``python -m implicit_gemm_gb300.build``);
loading raises if it is missing -- there is no other code path.

A problem spec is a dict: ndim, G, N, C, K, and per-dim lists in, filt,
stride, dil, pad_l, pad_r (ndim entries, outermost first), plus in_dtype
('bf16' | 'fp16') and out_dtype ('fp32' | 'bf16' | 'fp16').
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

DTYPES = {"bf16": 0, "fp16": 1, "fp32": 2}
MODES = {"auto": 0, "direct": 1, "atomic": 2, "deterministic": 3}
STATUS = {0: "WG_OK", 1: "WG_ERR_INVALID_ARGUMENT", 2: "WG_ERR_NOT_SUPPORTED", 3: "WG_ERR_MISALIGNED",
          4: "WG_ERR_WORKSPACE", 5: "WG_ERR_CUDA", 6: "WG_ERR_DEVICE_TIMEOUT", 7: "WG_ERR_INVALID_TOKEN",
          8: "WG_ERR_INVALID_OFFSET"}


class WgProblem(ctypes.Structure):
    _fields_ = [("ndim", ctypes.c_int), ("G", ctypes.c_int), ("N", ctypes.c_int), ("C", ctypes.c_int),
                ("K", ctypes.c_int), ("in_", ctypes.c_int * 3), ("filt", ctypes.c_int * 3),
                ("out", ctypes.c_int * 3), ("stride", ctypes.c_int * 3), ("dil", ctypes.c_int * 3),
                ("pad_l", ctypes.c_int * 3), ("pad_r", ctypes.c_int * 3), ("in_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int)]


class WgOptions(ctypes.Structure):
    _fields_ = [("split_k", ctypes.c_int), ("mode", ctypes.c_int), ("group_merge", ctypes.c_int),
                ("cluster", ctypes.c_int), ("kernel", ctypes.c_int)]


class WgMuonProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("ld", ctypes.c_longlong),
                ("batch_stride", ctypes.c_longlong), ("grad_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("weight_dtype", ctypes.c_int), ("steps", ctypes.c_int), ("nesterov", ctypes.c_int),
                ("coef", ctypes.POINTER(ctypes.c_float)), ("mu", ctypes.c_float), ("dampening", ctypes.c_float),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("lr", ctypes.c_float),
                ("weight_decay", ctypes.c_float)]


class WgEmbeddingProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_longlong), ("vocab", ctypes.c_int), ("dim", ctypes.c_int),
                ("ld_table", ctypes.c_longlong), ("ld_out", ctypes.c_longlong), ("table_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("token_bits", ctypes.c_int), ("padding_token", ctypes.c_int),
                ("scale", ctypes.c_float)]


class WgLinearProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_longlong), ("in_", ctypes.c_int), ("out", ctypes.c_int), ("experts", ctypes.c_int),
                ("ld_in", ctypes.c_longlong), ("ld_out", ctypes.c_longlong), ("ld_weight", ctypes.c_longlong),
                ("weight_stride", ctypes.c_longlong), ("ld_z", ctypes.c_longlong), ("ld_residual", ctypes.c_longlong),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("bias_dtype", ctypes.c_int),
                ("offset_bits", ctypes.c_int), ("activation", ctypes.c_int), ("dropout", ctypes.c_float),
                ("seed", ctypes.c_ulonglong), ("offset", ctypes.c_ulonglong), ("counter", ctypes.c_void_p)]


class WgActivationProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_longlong), ("dim", ctypes.c_int), ("ld_x", ctypes.c_longlong),
                ("ld_y", ctypes.c_longlong), ("ld_residual", ctypes.c_longlong), ("ld_dx", ctypes.c_longlong),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("bias_dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("dropout", ctypes.c_float), ("seed", ctypes.c_ulonglong),
                ("offset", ctypes.c_ulonglong), ("counter", ctypes.c_void_p)]


class WgradError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


EXPORTS = ("wg_problem_normalize", "wg_workspace_size", "wg_conv_bwd_weight", "wg_check_status",
           "wg_plan_string", "wg_status_string", "wg_last_error", "wg_conv_bwd_weight_noalloc",
           "wg_set_mark_event", "wg_conv_bwd_data", "wg_bwd_data_plan_string", "wg_bwd_data_workspace_size",
           "wg_conv_bwd_weight_host", "wg_selftest_timeout", "wg_muon_workspace_size", "wg_muon_plan_string",
           "wg_muon_update", "wg_embedding_lookup", "wg_embedding_workspace_size", "wg_embedding_bwd_weight",
           "wg_linear_workspace_size", "wg_linear_plan_string", "wg_linear", "wg_linear_bwd_data", "wg_linear_bwd_weight",
           "wg_activation_workspace_size", "wg_activation", "wg_activation_bwd")

_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load():
    """Load libwgrad.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"libwgrad.so not found at {_build.LIB}; build it with "
                                   "`python -m implicit_gemm_gb300.build` (needs nvcc)")
            lib = ctypes.CDLL(_build.LIB)
            P, O = ctypes.POINTER(WgProblem), ctypes.POINTER(WgOptions)
            lib.wg_problem_normalize.argtypes = [P]
            lib.wg_workspace_size.argtypes = [P, O, ctypes.POINTER(ctypes.c_size_t)]
            lib.wg_conv_bwd_weight.argtypes = [P, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, O,
                                               ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
            lib.wg_conv_bwd_weight_noalloc.argtypes = [P, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, O,
                                                       ctypes.c_void_p]
            lib.wg_conv_bwd_weight_host.argtypes = [P] + [ctypes.c_void_p] * 6 + [O, ctypes.c_void_p, ctypes.c_size_t,
                                                                                  ctypes.c_void_p]
            lib.wg_check_status.argtypes = [ctypes.c_void_p]
            lib.wg_selftest_timeout.argtypes = [ctypes.c_void_p]
            lib.wg_set_mark_event.argtypes = [ctypes.c_void_p]
            lib.wg_conv_bwd_data.argtypes = [P, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_size_t, ctypes.c_void_p]
            lib.wg_bwd_data_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
            lib.wg_bwd_data_plan_string.argtypes = [P, ctypes.c_char_p, ctypes.c_size_t]
            lib.wg_plan_string.argtypes = [P, O, ctypes.c_char_p, ctypes.c_size_t]
            MP, EP = ctypes.POINTER(WgMuonProblem), ctypes.POINTER(WgEmbeddingProblem)
            lib.wg_muon_workspace_size.argtypes = [MP, ctypes.POINTER(ctypes.c_size_t)]
            lib.wg_muon_plan_string.argtypes = [MP, ctypes.c_char_p, ctypes.c_size_t]
            lib.wg_muon_update.argtypes = [MP] + [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]
            lib.wg_embedding_lookup.argtypes = [EP] + [ctypes.c_void_p] * 4
            lib.wg_embedding_workspace_size.argtypes = [EP, ctypes.POINTER(ctypes.c_size_t)]
            lib.wg_embedding_bwd_weight.argtypes = [EP] + [ctypes.c_void_p] * 3 + [ctypes.c_int, ctypes.c_void_p,
                                                                                   ctypes.c_size_t, ctypes.c_void_p]
            LP, AP, V = ctypes.POINTER(WgLinearProblem), ctypes.POINTER(WgActivationProblem), ctypes.c_void_p
            lib.wg_linear_workspace_size.argtypes = [LP, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
            lib.wg_linear_plan_string.argtypes = [LP, ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]
            lib.wg_linear.argtypes = [LP] + [V] * 8 + [ctypes.c_size_t, V]
            lib.wg_linear_bwd_data.argtypes = [LP] + [V] * 7 + [ctypes.c_size_t, V]
            lib.wg_linear_bwd_weight.argtypes = [LP] + [V] * 5 + [ctypes.c_int, V, ctypes.c_size_t, V]
            lib.wg_activation_workspace_size.argtypes = [AP, ctypes.POINTER(ctypes.c_size_t)]
            lib.wg_activation.argtypes = [AP] + [V] * 5
            lib.wg_activation_bwd.argtypes = [AP] + [V] * 6 + [ctypes.c_size_t, V]
            lib.wg_status_string.argtypes = [ctypes.c_int]
            lib.wg_status_string.restype = ctypes.c_char_p
            lib.wg_last_error.restype = ctypes.c_char_p
            for name in EXPORTS:
                if name not in ("wg_status_string", "wg_last_error"):
                    getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def _check(st: int):
    if st != 0:
        raise WgradError(st, load().wg_last_error().decode())


def make_problem(spec: dict) -> WgProblem:
    p = WgProblem()
    nd = spec["ndim"]
    p.ndim, p.G, p.N, p.C, p.K = nd, spec["G"], spec["N"], spec["C"], spec["K"]
    for key, field, default in (("in", "in_", 1), ("filt", "filt", 1), ("stride", "stride", 1),
                                ("dil", "dil", 1), ("pad_l", "pad_l", 0), ("pad_r", "pad_r", 0),
                                ("out", "out", 0)):
        vals = list(spec.get(key, [default] * max(nd, 0)))
        arr = getattr(p, field)
        for i in range(3):
            arr[i] = vals[i] if i < min(nd, len(vals)) else 0
    p.in_dtype = DTYPES[spec.get("in_dtype", "bf16")]
    p.out_dtype = DTYPES[spec.get("out_dtype", "fp32")]
    return p


KERNELS = {"auto": 0, "igemm": 1, "depthwise": 2, "igemm_taps_m": 3, "igemm_taps_mn": 4, "igemm_pair": 5}


def make_options(split_k: int = 0, mode: str = "auto", group_merge: int = 0, cluster: int = 0,
                 kernel: str = "auto") -> WgOptions:
    return WgOptions(int(split_k), MODES[mode], int(group_merge), int(cluster), KERNELS[kernel])


def _addr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def wg_problem_normalize(spec: dict) -> list:
    """Derived output lengths (ndim entries)."""
    p = make_problem(spec)
    _check(load().wg_problem_normalize(ctypes.byref(p)))
    return [p.out[i] for i in range(spec["ndim"])]


def wg_workspace_size(spec: dict, split_k: int = 0, mode: str = "auto", group_merge: int = 0, *,
                      cluster: int = 0, kernel: str = "auto") -> int:
    p, o, n = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel), ctypes.c_size_t(0)
    _check(load().wg_workspace_size(ctypes.byref(p), ctypes.byref(o), ctypes.byref(n)))
    return int(n.value)


def wg_plan_string(spec: dict, split_k: int = 0, mode: str = "auto", group_merge: int = 0, *,
                   cluster: int = 0, kernel: str = "auto") -> str:
    p, o = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel)
    buf = ctypes.create_string_buffer(2048)
    _check(load().wg_plan_string(ctypes.byref(p), ctypes.byref(o), buf, len(buf)))
    return buf.value.decode()


def wg_conv_bwd_weight(spec: dict, x, dy, dw, split_k: int = 0, mode: str = "auto", group_merge: int = 0,
                       workspace=None, ws_bytes: int | None = None, stream=None, *, cluster: int = 0, kernel: str = "auto") -> None:
    """Launch the weight gradient on `stream` (torch stream, raw handle int, or None for
    torch's current stream when torch is loaded, else the legacy default stream)."""
    p, o = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel)
    if ws_bytes is None:
        ws_bytes = 0 if workspace is None else (workspace.numel() * workspace.element_size()
                                                if hasattr(workspace, "numel") else 0)
    _check(load().wg_conv_bwd_weight(ctypes.byref(p), _addr(x), _addr(dy), _addr(dw), ctypes.byref(o),
                                     _addr(workspace), int(ws_bytes), _stream_handle(stream)))


class PreparedCall:
    """wg_conv_bwd_weight with its arguments marshalled once: calling it makes one
    ctypes call.  Keeps references to the tensors it was built from."""

    def __init__(self, spec: dict, x, dy, dw, split_k: int = 0, mode: str = "auto", group_merge: int = 0,
                 workspace=None, ws_bytes: int | None = None, *, cluster: int = 0, kernel: str = "auto"):
        self._keep = (x, dy, dw, workspace)
        self.p, self.o = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel)
        if ws_bytes is None:
            ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        self.fn = load().wg_conv_bwd_weight
        self.args = (ctypes.byref(self.p), ctypes.c_void_p(_addr(x)), ctypes.c_void_p(_addr(dy)),
                     ctypes.c_void_p(_addr(dw)), ctypes.byref(self.o), ctypes.c_void_p(_addr(workspace)),
                     ctypes.c_size_t(int(ws_bytes)))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


def wg_conv_bwd_weight_host(spec: dict, x_host, dy_host, dw_host, x_dev, dy_dev, dw_dev, split_k: int = 0,
                            mode: str = "auto", group_merge: int = 0, workspace=None, ws_bytes: int | None = None,
                            stream=None, *, cluster: int = 0, kernel: str = "auto") -> None:
    """The weight gradient from host buffers (x_host, dy_host; ideally pinned) into dw_host,
    staged through the device buffers x_dev, dy_dev, dw_dev; copies overlap the compute."""
    p, o = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel)
    if ws_bytes is None:
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().wg_conv_bwd_weight_host(ctypes.byref(p), _addr(x_host), _addr(dy_host), _addr(dw_host),
                                          _addr(x_dev), _addr(dy_dev), _addr(dw_dev), ctypes.byref(o),
                                          _addr(workspace), int(ws_bytes), _stream_handle(stream)))


class PreparedHostCall:
    """wg_conv_bwd_weight_host with its arguments marshalled once (one ctypes call per use)."""

    def __init__(self, spec: dict, x_host, dy_host, dw_host, x_dev, dy_dev, dw_dev, split_k: int = 0,
                 mode: str = "auto", group_merge: int = 0, workspace=None, ws_bytes: int | None = None, *,
                 cluster: int = 0, kernel: str = "auto"):
        self._keep = (x_host, dy_host, dw_host, x_dev, dy_dev, dw_dev, workspace)
        self.p, self.o = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel)
        if ws_bytes is None:
            ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        self.fn = load().wg_conv_bwd_weight_host
        self.args = (ctypes.byref(self.p), *(ctypes.c_void_p(_addr(t)) for t in (x_host, dy_host, dw_host, x_dev,
                                                                                 dy_dev, dw_dev)),
                     ctypes.byref(self.o), ctypes.c_void_p(_addr(workspace)), ctypes.c_size_t(int(ws_bytes)))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


def wg_conv_bwd_weight_noalloc(spec: dict, x, dy, dw, split_k: int = 0, mode: str = "auto", group_merge: int = 0,
                               stream=None, *, cluster: int = 0, kernel: str = "auto") -> None:
    """wg_conv_bwd_weight for callers that cannot allocate: the split-K workspace comes
    from the library's own 16 MiB device array (see include/wgrad.h)."""
    p, o = make_problem(spec), make_options(split_k, mode, group_merge, cluster, kernel)
    _check(load().wg_conv_bwd_weight_noalloc(ctypes.byref(p), _addr(x), _addr(dy), _addr(dw), ctypes.byref(o),
                                             _stream_handle(stream)))


def wg_conv_bwd_data(spec: dict, dy, w, dx, workspace=None, ws_bytes: int | None = None, stream=None) -> None:
    """Backward-data: dX (spec's out_dtype) from dY and W (spec's in_dtype); see include/wgrad.h."""
    p = make_problem(spec)
    if ws_bytes is None:
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().wg_conv_bwd_data(ctypes.byref(p), _addr(dy), _addr(w), _addr(dx), _addr(workspace), int(ws_bytes),
                                   _stream_handle(stream)))


def wg_bwd_data_workspace_size(spec: dict) -> int:
    p, n = make_problem(spec), ctypes.c_size_t(0)
    _check(load().wg_bwd_data_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def wg_bwd_data_plan_string(spec: dict) -> str:
    p = make_problem(spec)
    buf = ctypes.create_string_buffer(1024)
    _check(load().wg_bwd_data_plan_string(ctypes.byref(p), buf, len(buf)))
    return buf.value.decode()


class PreparedDgradCall:
    """wg_conv_bwd_data with its arguments marshalled once."""

    def __init__(self, spec: dict, dy, w, dx, workspace=None, ws_bytes: int = 0):
        self._keep = (dy, w, dx, workspace)
        self.p = make_problem(spec)
        self.fn = load().wg_conv_bwd_data
        self.args = (ctypes.byref(self.p), ctypes.c_void_p(_addr(dy)), ctypes.c_void_p(_addr(w)),
                     ctypes.c_void_p(_addr(dx)), ctypes.c_void_p(_addr(workspace)), ctypes.c_size_t(int(ws_bytes)))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


def conv_bwd_data(spec: dict, dy, w, out=None, stream=None):
    """Convenience wrapper over wg_conv_bwd_data for torch CUDA tensors: allocates dX
    (N, *in, G, C) in spec['out_dtype'] with torch, then calls the library."""
    import torch
    tdt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[spec.get("out_dtype", "fp32")]
    if out is None:
        out = _empty(stream, (spec["N"], *spec["in"], spec["G"], spec["C"]), tdt, dy.device, returned=True)
    nbytes = wg_bwd_data_workspace_size(spec)
    ws = _empty(stream, nbytes, torch.uint8, dy.device) if nbytes else None
    wg_conv_bwd_data(spec, dy, w, out, ws, nbytes, stream)
    return out


def wg_set_mark_event(event) -> None:
    """Record `event` (a torch.cuda.Event, a raw cudaEvent_t, or None to stop) after
    the main kernel of every following call from this thread (see include/wgrad.h).
    A torch event must have been recorded once, so that it exists."""
    h = None if event is None else (event if isinstance(event, int) else int(event.cuda_event))
    _check(load().wg_set_mark_event(h))


def wg_selftest_timeout(stream=None) -> None:
    """Launch the library's bounded-wait self-test (see include/wgrad.h)."""
    _check(load().wg_selftest_timeout(_stream_handle(stream)))


def wg_check_status(stream=None) -> None:
    _check(load().wg_check_status(_stream_handle(stream)))


def wg_status_string(status: int) -> str:
    return load().wg_status_string(int(status)).decode()


def wg_last_error() -> str:
    return load().wg_last_error().decode()


def _stream_handle(stream):
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available() and torch.cuda.is_initialized():
                return int(torch.cuda.current_stream().cuda_stream)
        except Exception:  # pragma: no cover - torch missing
            pass
        return None
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _empty(stream, shape, dtype, device, returned: bool = False):
    """torch.empty for a call on `stream` (None: the current one).  The memory comes from that stream's own blocks: one
    of the current stream's may still be in use by work that is pending there, which `stream` does not wait for.
    `returned`: the caller gets the tensor, so work on the current stream may use it too."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    on = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream_handle(stream), device)
    with torch.cuda.stream(on):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(here)
    return t


def _zeros(stream, shape, dtype, device, returned: bool = False):
    """The same, filled with zeros on the call's stream."""
    import torch
    t = _empty(stream, shape, dtype, device, returned)
    with torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream if isinstance(stream, torch.cuda.Stream)
                           else torch.cuda.ExternalStream(_stream_handle(stream), device)):
        t.zero_()
    return t


def conv_bwd_weight(spec: dict, x, dy, split_k: int = 0, mode: str = "auto", group_merge: int = 0, out=None,
                    stream=None, *, cluster: int = 0, kernel: str = "auto"):
    """Convenience wrapper over wg_conv_bwd_weight for torch CUDA tensors: allocates dW
    (G, K, *filt, C) in spec['out_dtype'] and the workspace it needs with torch, then calls
    the library."""
    import torch
    tdt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[spec.get("out_dtype", "fp32")]
    if out is None:
        out = _empty(stream, (spec["G"], spec["K"], *spec["filt"], spec["C"]), tdt, x.device, returned=True)
    nbytes = wg_workspace_size(spec, split_k, mode, group_merge, cluster=cluster, kernel=kernel)
    ws = _empty(stream, nbytes, torch.uint8, x.device) if nbytes else None
    wg_conv_bwd_weight(spec, x, dy, out, split_k, mode, group_merge, ws, nbytes, stream, cluster=cluster,
                       kernel=kernel)
    return out


# ---------------------------------------------------------------- weight updates

def make_muon_problem(spec: dict) -> WgMuonProblem:
    """A spec is a dict: batch (default 1), rows, cols, and optionally ld, batch_stride (elements; 0 = packed),
    grad_dtype, out_dtype, weight_dtype ('fp32' | 'bf16' | 'fp16'; defaults fp32, bf16, bf16), steps (5), coef (a list
    of one (a, b, c) per step), eps (1e-7), scale (1), momentum (0.95), dampening (0), nesterov (True), lr (0),
    weight_decay (0).  See include/wgrad.h for the formula."""
    p = WgMuonProblem()
    p.batch, p.rows, p.cols = spec.get("batch", 1), spec["rows"], spec["cols"]
    p.ld, p.batch_stride = spec.get("ld", 0), spec.get("batch_stride", 0)
    p.grad_dtype = DTYPES[spec.get("grad_dtype", "fp32")]
    p.out_dtype = DTYPES[spec.get("out_dtype", "bf16")]
    p.weight_dtype = DTYPES[spec.get("weight_dtype", "bf16")]
    p.steps, p.nesterov = spec.get("steps", 5), int(spec.get("nesterov", True))
    coef = spec.get("coef")
    if coef is not None:
        flat = [float(v) for step in coef for v in step]
        if len(flat) != 3 * max(p.steps, 0):
            raise ValueError("coef needs one (a, b, c) per step")
        p.coef = (ctypes.c_float * max(len(flat), 1))(*flat)
    p.mu, p.dampening = spec.get("momentum", 0.95), spec.get("dampening", 0.0)
    p.eps, p.scale = spec.get("eps", 1e-7), spec.get("scale", 1.0)
    p.lr, p.weight_decay = spec.get("lr", 0.0), spec.get("weight_decay", 0.0)
    return p


def _bytes_of(workspace, ws_bytes) -> int:
    if ws_bytes is not None:
        return int(ws_bytes)
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def wg_muon_workspace_size(spec: dict) -> int:
    p, n = make_muon_problem(spec), ctypes.c_size_t(0)
    _check(load().wg_muon_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def wg_muon_plan_string(spec: dict) -> str:
    p, buf = make_muon_problem(spec), ctypes.create_string_buffer(1024)
    _check(load().wg_muon_plan_string(ctypes.byref(p), buf, len(buf)))
    return buf.value.decode()


def wg_muon_update(spec: dict, grad, momentum=None, weight=None, out=None, workspace=None, ws_bytes: int | None = None,
                   stream=None) -> None:
    """The orthogonalised update of grad, with the momentum and the weight step where those are given."""
    p = make_muon_problem(spec)
    _check(load().wg_muon_update(ctypes.byref(p), _addr(grad), _addr(momentum), _addr(weight), _addr(out),
                                 _addr(workspace), _bytes_of(workspace, ws_bytes), _stream_handle(stream)))


class PreparedMuonUpdate:
    """wg_muon_update with its arguments marshalled once: calling it makes one ctypes call.  Keeps
    references to the tensors it was built from."""

    def __init__(self, spec: dict, grad, momentum=None, weight=None, out=None, workspace=None,
                 ws_bytes: int | None = None):
        self._keep = (grad, momentum, weight, out, workspace)
        self.p = make_muon_problem(spec)
        self.fn = load().wg_muon_update
        self.args = (ctypes.byref(self.p), *(ctypes.c_void_p(_addr(t)) for t in self._keep),
                     ctypes.c_size_t(_bytes_of(workspace, ws_bytes)))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


def _expect(name, t, dtype: str, shape=None, elements: int = 0) -> None:
    """Refuse a tensor that is not what the call will take it for: of `dtype`, contiguous and of `shape`, or (no shape)
    with `elements` elements from its first one on."""
    if t is None:
        return
    names = {"torch.float32": "fp32", "torch.bfloat16": "bf16", "torch.float16": "fp16"}
    if names.get(str(t.dtype)) != dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if shape is None:
        if t.untyped_storage().nbytes() // t.element_size() - t.storage_offset() < elements:
            raise ValueError(f"{name} holds fewer than {elements} elements")
    elif tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(**tensors) -> None:
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} is not a CUDA tensor")


def muon_update(spec: dict, grad, momentum=None, weight=None, out=None, stream=None):
    """Convenience wrapper over wg_muon_update for torch CUDA tensors: allocates the workspace, and `out` (grad's
    shape; with ld or batch_stride a (batch, rows, cols) view of that layout) when no weight is given, then calls the
    library.  Returns out, or the weight.  Tensors of another type or size than the spec's are refused."""
    import torch
    nbytes = wg_muon_workspace_size(spec)  # (checks the spec)
    b, rows, cols, ld, bs = (spec.get(k, 0) for k in ("batch", "rows", "cols", "ld", "batch_stride"))
    b, ld = b or 1, ld or cols
    span = (b - 1) * (bs or rows * ld) + (rows - 1) * ld + cols
    made = out is None and weight is None
    types = {"grad": spec.get("grad_dtype", "fp32"), "momentum": "fp32", "weight": spec.get("weight_dtype", "bf16"),
             "out": spec.get("out_dtype", "bf16")}
    for name, t in (("grad", grad), ("momentum", momentum), ("weight", weight), ("out", out)):
        _expect(name, t, types[name], elements=span)
        if t is not None and not (spec.get("ld", 0) or bs) and not (t.is_contiguous() and t.numel() == span):
            raise ValueError(f"{name} must be contiguous, of batch * rows * cols elements")
    _on_gpu(grad=grad, momentum=momentum, weight=weight, out=out)
    if made:
        tdt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[types["out"]]
        if spec.get("ld", 0) or bs:
            out = _empty(stream, span, tdt, grad.device, returned=True).as_strided((b, rows, cols), (bs or rows * ld, ld, 1))
        else:
            out = _empty(stream, grad.shape, tdt, grad.device, returned=True)
    ws = _empty(stream, max(nbytes, 1), torch.uint8, grad.device)
    wg_muon_update(spec, grad, momentum, weight, out, ws, nbytes, stream)
    return out if out is not None else weight


def make_embedding_problem(spec: dict) -> WgEmbeddingProblem:
    """A spec is a dict: tokens, vocab, dim, and optionally ld_table, ld_out (elements; 0 = dim), table_dtype,
    out_dtype ('fp32' | 'bf16' | 'fp16'; default bf16), token_dtype ('i32' | 'i64'; default i64), scale (1),
    padding_token (-1 = none)."""
    p = WgEmbeddingProblem()
    p.tokens, p.vocab, p.dim = spec["tokens"], spec["vocab"], spec["dim"]
    p.ld_table, p.ld_out = spec.get("ld_table", 0), spec.get("ld_out", 0)
    p.table_dtype = DTYPES[spec.get("table_dtype", "bf16")]
    p.out_dtype = DTYPES[spec.get("out_dtype", "bf16")]
    p.token_bits = {"i32": 32, "i64": 64}[spec.get("token_dtype", "i64")]
    p.padding_token, p.scale = spec.get("padding_token", -1), spec.get("scale", 1.0)
    return p


def wg_embedding_lookup(spec: dict, token, table, out, stream=None) -> None:
    """out[t] = scale * table[token[t]]."""
    p = make_embedding_problem(spec)
    _check(load().wg_embedding_lookup(ctypes.byref(p), _addr(token), _addr(table), _addr(out), _stream_handle(stream)))


def wg_embedding_workspace_size(spec: dict) -> int:
    p, n = make_embedding_problem(spec), ctypes.c_size_t(0)
    _check(load().wg_embedding_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def wg_embedding_bwd_weight(spec: dict, token, dy, dtable, accumulate: bool = False, workspace=None,
                            ws_bytes: int | None = None, stream=None) -> None:
    """dtable[v] = (accumulate ? dtable[v] : 0) + scale * sum of dy[t] over the t with token[t] = v."""
    p = make_embedding_problem(spec)
    _check(load().wg_embedding_bwd_weight(ctypes.byref(p), _addr(token), _addr(dy), _addr(dtable), int(accumulate),
                                          _addr(workspace), _bytes_of(workspace, ws_bytes), _stream_handle(stream)))


class PreparedEmbeddingLookup:
    """wg_embedding_lookup with its arguments marshalled once."""

    def __init__(self, spec: dict, token, table, out):
        self._keep = (token, table, out)
        self.p = make_embedding_problem(spec)
        self.fn = load().wg_embedding_lookup
        self.args = (ctypes.byref(self.p), *(ctypes.c_void_p(_addr(t)) for t in self._keep))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


class PreparedEmbeddingBwd:
    """wg_embedding_bwd_weight with its arguments marshalled once."""

    def __init__(self, spec: dict, token, dy, dtable, accumulate: bool = False, workspace=None,
                 ws_bytes: int | None = None):
        self._keep = (token, dy, dtable, workspace)
        self.p = make_embedding_problem(spec)
        self.fn = load().wg_embedding_bwd_weight
        self.args = (ctypes.byref(self.p), *(ctypes.c_void_p(_addr(t)) for t in (token, dy, dtable)),
                     ctypes.c_int(int(accumulate)), ctypes.c_void_p(_addr(workspace)),
                     ctypes.c_size_t(_bytes_of(workspace, ws_bytes)))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


def _embedding_spec(token, vocab, dim, table_dtype, out_dtype, scale, padding_token):
    names = {"torch.float32": "fp32", "torch.bfloat16": "bf16", "torch.float16": "fp16"}
    tokens = {"torch.int32": "i32", "torch.int64": "i64"}
    if str(token.dtype) not in tokens or not token.is_contiguous():
        raise ValueError("token must be a contiguous int32 or int64 tensor")
    for t in (table_dtype, out_dtype):
        if str(t) not in names:
            raise ValueError(f"{t} is not supported")
    return {"tokens": token.numel(), "vocab": vocab, "dim": dim, "table_dtype": names[str(table_dtype)],
            "out_dtype": names[str(out_dtype)], "token_dtype": tokens[str(token.dtype)], "scale": scale,
            "padding_token": padding_token}


def embedding_lookup(token, table, scale: float = 1.0, out=None, stream=None):
    """Convenience wrapper over wg_embedding_lookup for torch CUDA tensors: contiguous int32 or int64 tokens of any
    shape, a contiguous (vocab, dim) table.  Returns (*token.shape, dim) in table's dtype (or `out`)."""
    vocab, dim = table.shape
    made = out is None
    spec = _embedding_spec(token, vocab, dim, table.dtype, table.dtype if made else out.dtype, scale, -1)
    _expect("table", table, spec["table_dtype"], (vocab, dim))
    _expect("out", out, spec["out_dtype"], (*token.shape, dim))
    _on_gpu(token=token, table=table, out=out)
    if made:
        out = _empty(stream, (*token.shape, dim), table.dtype, table.device, returned=True)
    wg_embedding_lookup(spec, token, table, out, stream)
    return out


def embedding_bwd_weight(token, dy, vocab: int, scale: float = 1.0, padding_token: int = -1, out=None,
                         accumulate: bool = False, stream=None):
    """Convenience wrapper over wg_embedding_bwd_weight for torch CUDA tensors: contiguous dy of shape
    (*token.shape, dim).  Returns the (vocab, dim) gradient in dy's dtype (or `out`, added to when accumulate)."""
    import torch
    made, dim = out is None, dy.shape[-1]
    if made and accumulate:
        raise ValueError("accumulate needs out")
    spec = _embedding_spec(token, vocab, dim, dy.dtype if made else out.dtype, dy.dtype, scale, padding_token)
    nbytes = wg_embedding_workspace_size(spec)  # (checks the spec)
    _expect("dy", dy, spec["out_dtype"], (*token.shape, dim))
    _expect("out", out, spec["table_dtype"], (vocab, dim))
    _on_gpu(token=token, dy=dy, out=out)
    if made:
        out = _empty(stream, (vocab, dim), dy.dtype, dy.device, returned=True)
    ws = _empty(stream, max(nbytes, 1), torch.uint8, dy.device)
    wg_embedding_bwd_weight(spec, token, dy, out, accumulate, ws, nbytes, stream)
    return out


# ---------------------------------------------------------------- layers

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LINEAR_CALLS = {"forward": 0, "bwd_data": 1, "bwd_weight": 2}


def _set_tail(p, spec: dict) -> None:
    p.in_dtype, p.out_dtype = DTYPES[spec.get("in_dtype", "bf16")], DTYPES[spec.get("out_dtype", "bf16")]
    p.bias_dtype = DTYPES[spec.get("bias_dtype", "fp32")]
    p.activation, p.dropout = ACTIVATIONS[spec.get("activation", "none")], spec.get("dropout", 0.0)
    p.seed, p.offset = int(spec.get("seed", 0)) % (1 << 64), int(spec.get("offset", 0)) % (1 << 64)
    p.counter = _addr(spec.get("counter")) or None


def make_linear_problem(spec: dict) -> WgLinearProblem:
    """A spec is a dict: tokens, in, out, and optionally experts (0), ld_in, ld_out, ld_weight, weight_stride, ld_z,
    ld_residual (elements; 0 = packed), in_dtype, out_dtype ('bf16'), bias_dtype ('fp32'), offset_dtype ('i32' | 'i64',
    default i32), activation ('none' | 'relu' | 'gelu' | 'gelu_tanh' | 'silu'), dropout (0), seed, offset (0), counter (a
    device tensor of one 64-bit integer, or None; the caller keeps it).  See include/wgrad.h for the formulas."""
    p = WgLinearProblem()
    p.tokens, p.in_, p.out, p.experts = spec["tokens"], spec["in"], spec["out"], spec.get("experts", 0)
    for key in ("ld_in", "ld_out", "ld_weight", "weight_stride", "ld_z", "ld_residual"):
        setattr(p, key, spec.get(key, 0))
    p.offset_bits = {"i32": 32, "i64": 64}[spec.get("offset_dtype", "i32")]
    _set_tail(p, spec)
    return p


def make_activation_problem(spec: dict) -> WgActivationProblem:
    """A spec is a dict: tokens, dim, and optionally ld_x, ld_y, ld_residual, ld_dx (elements; 0 = dim), in_dtype,
    out_dtype ('bf16'), bias_dtype ('fp32'), activation, dropout, seed, offset, counter (as in make_linear_problem)."""
    p = WgActivationProblem()
    p.tokens, p.dim = spec["tokens"], spec["dim"]
    for key in ("ld_x", "ld_y", "ld_residual", "ld_dx"):
        setattr(p, key, spec.get(key, 0))
    _set_tail(p, spec)
    return p


def wg_linear_workspace_size(spec: dict, call: str = "forward") -> int:
    """Bytes of workspace of a call: 'forward', 'bwd_data' or 'bwd_weight'."""
    p, n = make_linear_problem(spec), ctypes.c_size_t(0)
    _check(load().wg_linear_workspace_size(ctypes.byref(p), LINEAR_CALLS[call], ctypes.byref(n)))
    return int(n.value)


def wg_linear_plan_string(spec: dict, call: str = "forward") -> str:
    p, buf = make_linear_problem(spec), ctypes.create_string_buffer(1024)
    _check(load().wg_linear_plan_string(ctypes.byref(p), LINEAR_CALLS[call], buf, len(buf)))
    return buf.value.decode()


def wg_activation_workspace_size(spec: dict) -> int:
    p, n = make_activation_problem(spec), ctypes.c_size_t(0)
    _check(load().wg_activation_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


class _Prepared:
    """A call with its arguments marshalled once: calling it makes one ctypes call.  Keeps references to the tensors it
    was built from.  `p` is the problem record: a change to it (p.offset of a dropout, say) counts for later calls."""

    def _set(self, fn, p, tensors, extra, keep, workspace, ws_bytes, has_workspace=True):
        self._keep = (*tensors, workspace, keep)
        self.p, self.fn = p, fn
        self.args = (ctypes.byref(p), *(ctypes.c_void_p(_addr(t)) for t in tensors), *extra)
        if has_workspace:
            self.args += (ctypes.c_void_p(_addr(workspace)), ctypes.c_size_t(_bytes_of(workspace, ws_bytes)))

    def __call__(self, stream_handle: int | None = None) -> None:
        st = self.fn(*self.args, stream_handle)
        if st:
            _check(st)


class PreparedLinear(_Prepared):
    """wg_linear with its arguments marshalled once."""

    def __init__(self, spec: dict, x, w, y, bias=None, residual=None, z=None, offsets=None, workspace=None,
                 ws_bytes: int | None = None):
        self._set(load().wg_linear, make_linear_problem(spec), (offsets, x, w, bias, residual, y, z), (), spec.get("counter"),
                  workspace, ws_bytes)


class PreparedLinearBwdData(_Prepared):
    """wg_linear_bwd_data with its arguments marshalled once."""

    def __init__(self, spec: dict, dy, w, dx, z=None, residual=None, offsets=None, workspace=None, ws_bytes: int | None = None):
        self._set(load().wg_linear_bwd_data, make_linear_problem(spec), (offsets, dy, w, z, residual, dx), (),
                  spec.get("counter"), workspace, ws_bytes)


class PreparedLinearBwdWeight(_Prepared):
    """wg_linear_bwd_weight with its arguments marshalled once."""

    def __init__(self, spec: dict, x, dy, dw, dbias=None, accumulate: bool = False, offsets=None, workspace=None,
                 ws_bytes: int | None = None):
        self._set(load().wg_linear_bwd_weight, make_linear_problem(spec), (offsets, x, dy, dw, dbias),
                  (ctypes.c_int(int(accumulate)),), spec.get("counter"), workspace, ws_bytes)


class PreparedActivation(_Prepared):
    """wg_activation with its arguments marshalled once."""

    def __init__(self, spec: dict, x, y, bias=None, residual=None):
        self._set(load().wg_activation, make_activation_problem(spec), (x, bias, residual, y), (), spec.get("counter"), None, 0,
                  False)


class PreparedActivationBwd(_Prepared):
    """wg_activation_bwd with its arguments marshalled once."""

    def __init__(self, spec: dict, dy, x, dx, bias=None, dbias=None, workspace=None, ws_bytes: int | None = None):
        self._set(load().wg_activation_bwd, make_activation_problem(spec), (dy, x, bias, dx, dbias), (), spec.get("counter"),
                  workspace, ws_bytes)


def wg_linear(spec: dict, x, w, y, bias=None, residual=None, z=None, offsets=None, workspace=None, ws_bytes: int | None = None,
              stream=None) -> None:
    """y = residual + D(act(x w' + bias)), z the pre-activations where given; by expert where the spec has experts."""
    PreparedLinear(spec, x, w, y, bias, residual, z, offsets, workspace, ws_bytes)(_stream_handle(stream))


def wg_linear_bwd_data(spec: dict, dy, w, dx, z=None, residual=None, offsets=None, workspace=None, ws_bytes: int | None = None,
                       stream=None) -> None:
    """dx = residual + D(act'(z) (dy w))."""
    PreparedLinearBwdData(spec, dy, w, dx, z, residual, offsets, workspace, ws_bytes)(_stream_handle(stream))


def wg_linear_bwd_weight(spec: dict, x, dy, dw, dbias=None, accumulate: bool = False, offsets=None, workspace=None,
                         ws_bytes: int | None = None, stream=None) -> None:
    """dw = dy' x and dbias = column sums of dy, per expert; added to what is there when accumulate."""
    PreparedLinearBwdWeight(spec, x, dy, dw, dbias, accumulate, offsets, workspace, ws_bytes)(_stream_handle(stream))


def wg_activation(spec: dict, x, y, bias=None, residual=None, stream=None) -> None:
    """y = residual + D(act(x + bias))."""
    PreparedActivation(spec, x, y, bias, residual)(_stream_handle(stream))


def wg_activation_bwd(spec: dict, dy, x, dx, bias=None, dbias=None, workspace=None, ws_bytes: int | None = None,
                      stream=None) -> None:
    """dx = D(act'(x + bias) dy), dbias = column sums of dx."""
    PreparedActivationBwd(spec, dy, x, dx, bias, dbias, workspace, ws_bytes)(_stream_handle(stream))


_NAMES = {"torch.float32": "fp32", "torch.bfloat16": "bf16", "torch.float16": "fp16"}


def _name(t, what: str) -> str:
    if str(t) not in _NAMES:
        raise ValueError(f"{what} of type {t} is not supported")
    return _NAMES[str(t)]


def _tail_spec(activation, dropout, seed, offset, counter) -> dict:
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {', '.join(ACTIVATIONS)}")
    if counter is not None and (str(counter.dtype) != "torch.int64" or counter.numel() != 1):
        raise ValueError("counter must be an int64 tensor of one element")
    _on_gpu(counter=counter)
    return {"activation": activation, "dropout": dropout, "seed": seed, "offset": offset, "counter": counter}


def _same_device(**tensors) -> None:
    _on_gpu(**tensors)
    devices = {t.device for t in tensors.values() if t is not None}
    if len(devices) > 1:
        raise ValueError("tensors on different devices: " + ", ".join(sorted(map(str, devices))))


def _linear_spec(rows, w, offsets, in_dtype, out_dtype, bias, tail) -> dict:
    """Of x or dy's rows and w (or the weight gradient's shape): (out, in), or (experts, out, in) with offsets."""
    shape = tuple(w)
    if len(shape) != (2 if offsets is None else 3):
        raise ValueError("w must have shape (out, in), or (experts, out, in) with offsets")
    experts = 0 if offsets is None else shape[0]
    spec = {"tokens": rows, "in": shape[-1], "out": shape[-2], "experts": experts, "in_dtype": in_dtype, "out_dtype": out_dtype,
            "bias_dtype": "fp32" if bias is None else _name(bias.dtype, "a bias"), **tail}
    if offsets is not None:
        kinds = {"torch.int32": "i32", "torch.int64": "i64"}
        if str(offsets.dtype) not in kinds or not offsets.is_contiguous() or offsets.numel() != experts + 1:
            raise ValueError("offsets must be contiguous int32 or int64, one more than experts")
        spec["offset_dtype"] = kinds[str(offsets.dtype)]
    return spec


def linear(x, w, bias=None, residual=None, activation: str = "none", dropout: float = 0.0, seed: int = 0, offset: int = 0,
           counter=None, offsets=None, keep_z: bool = False, out=None, stream=None):
    """Convenience wrapper over wg_linear for contiguous torch CUDA tensors: x of shape (..., in), w (out, in) and bias
    (out,), or with offsets (experts + 1 row numbers) x (rows, in), w (experts, out, in) and bias (experts, out).  Returns
    y of shape (..., out) in x's type (or residual's, or `out`), or (y, z) when keep_z.  Without `out`, rows of no expert
    are zeros."""
    import torch
    dt = _name(x.dtype, "x")
    ydt = out.dtype if out is not None else residual.dtype if residual is not None else x.dtype
    rows = x.numel() // x.shape[-1] if x.shape[-1] else 0
    spec = _linear_spec(rows, w.shape, offsets, dt, _name(ydt, "y"), bias, _tail_spec(activation, dropout, seed, offset, counter))
    nbytes = wg_linear_workspace_size(spec, "forward")  # (checks the spec)
    shape = (*x.shape[:-1], spec["out"])
    _expect("x", x, dt, (*x.shape[:-1], spec["in"]))
    _expect("w", w, dt, w.shape)
    _expect("bias", bias, spec["bias_dtype"], w.shape[:-1])
    _expect("residual", residual, spec["out_dtype"], shape)
    _expect("out", out, spec["out_dtype"], shape)
    _same_device(x=x, w=w, bias=bias, residual=residual, out=out, offsets=offsets, counter=counter)
    with torch.cuda.device(x.device):
        make = _zeros if offsets is not None else _empty
        z = make(stream, shape, x.dtype, x.device, returned=True) if keep_z else None
        if out is None:
            out = make(stream, shape, ydt, x.device, returned=True)
        ws = _empty(stream, nbytes, torch.uint8, x.device)
        wg_linear(spec, x, w, out, bias, residual, z, offsets, ws, nbytes, stream)
    return (out, z) if keep_z else out


def linear_bwd_data(dy, w, z=None, residual=None, activation: str = "none", dropout: float = 0.0, seed: int = 0, offset: int = 0,
                    counter=None, offsets=None, out=None, stream=None):
    """Convenience wrapper over wg_linear_bwd_data: dy (..., out), w as in linear; z (..., in) and the factors of the layer
    below where its activation and dropout made x.  Returns dx (..., in) in dy's type (or residual's, or `out`)."""
    import torch
    dt = _name(dy.dtype, "dy")
    xdt = out.dtype if out is not None else residual.dtype if residual is not None else dy.dtype
    rows = dy.numel() // dy.shape[-1] if dy.shape[-1] else 0
    spec = _linear_spec(rows, w.shape, offsets, dt, _name(xdt, "dx"), None, _tail_spec(activation, dropout, seed, offset, counter))
    nbytes = wg_linear_workspace_size(spec, "bwd_data")
    shape = (*dy.shape[:-1], spec["in"])
    _expect("dy", dy, dt, (*dy.shape[:-1], spec["out"]))
    _expect("w", w, dt, w.shape)
    _expect("z", z, dt, shape)
    _expect("residual", residual, spec["out_dtype"], shape)
    _expect("out", out, spec["out_dtype"], shape)
    _same_device(dy=dy, w=w, z=z, residual=residual, out=out, offsets=offsets, counter=counter)
    with torch.cuda.device(dy.device):
        if out is None:
            out = (_zeros if offsets is not None else _empty)(stream, shape, xdt, dy.device, returned=True)
        ws = _empty(stream, nbytes, torch.uint8, dy.device)
        wg_linear_bwd_data(spec, dy, w, out, z, residual, offsets, ws, nbytes, stream)
    return out


def linear_bwd_weight(x, dy, offsets=None, out=None, dbias=None, accumulate: bool = False, stream=None):
    """Convenience wrapper over wg_linear_bwd_weight: x (..., in), dy (..., out).  Returns dw (out, in), or (experts, out,
    in) with offsets, fp32 (or `out`, added to when accumulate).  dbias ((out,) or (experts, out)) is written where given."""
    import torch
    dt = _name(x.dtype, "x")
    if out is None and accumulate:
        raise ValueError("accumulate needs out")
    shape = (dy.shape[-1], x.shape[-1]) if offsets is None else (offsets.numel() - 1, dy.shape[-1], x.shape[-1])
    rows = x.numel() // x.shape[-1] if x.shape[-1] else 0
    wdt = torch.float32 if out is None else out.dtype
    spec = _linear_spec(rows, shape, offsets, dt, _name(wdt, "dw"), dbias, {})
    nbytes = wg_linear_workspace_size(spec, "bwd_weight")
    _expect("x", x, dt, (*x.shape[:-1], spec["in"]))
    _expect("dy", dy, dt, (*x.shape[:-1], spec["out"]))
    _expect("out", out, spec["out_dtype"], shape)
    _expect("dbias", dbias, spec["bias_dtype"], shape[:-1])
    _same_device(x=x, dy=dy, out=out, dbias=dbias, offsets=offsets)
    with torch.cuda.device(x.device):
        if out is None:
            out = _empty(stream, shape, wdt, x.device, returned=True)
        ws = _empty(stream, nbytes, torch.uint8, x.device)
        wg_linear_bwd_weight(spec, x, dy, out, dbias, accumulate, offsets, ws, nbytes, stream)
    return out


def activation(x, bias=None, residual=None, activation: str = "none", dropout: float = 0.0, seed: int = 0, offset: int = 0,
               counter=None, out=None, stream=None):
    """Convenience wrapper over wg_activation for contiguous torch CUDA tensors: residual + D(act(x + bias)), x of shape
    (..., dim).  Returns y in x's type (or residual's, or `out`, which may be x or residual)."""
    import torch
    ydt = out.dtype if out is not None else residual.dtype if residual is not None else x.dtype
    dim = x.shape[-1]
    spec = {"tokens": x.numel() // dim if dim else 0, "dim": dim, "in_dtype": _name(x.dtype, "x"), "out_dtype": _name(ydt, "y"),
            "bias_dtype": "fp32" if bias is None else _name(bias.dtype, "bias"),
            **_tail_spec(activation, dropout, seed, offset, counter)}
    wg_activation_workspace_size(spec)  # (checks the spec)
    _expect("x", x, spec["in_dtype"], x.shape)
    _expect("bias", bias, spec["bias_dtype"], (dim,))
    _expect("residual", residual, spec["out_dtype"], x.shape)
    _expect("out", out, spec["out_dtype"], x.shape)
    _same_device(x=x, bias=bias, residual=residual, out=out, counter=counter)
    with torch.cuda.device(x.device):
        if out is None:
            out = _empty(stream, x.shape, ydt, x.device, returned=True)
        wg_activation(spec, x, out, bias, residual, stream)
    return out


def activation_bwd(dy, x=None, bias=None, activation: str = "none", dropout: float = 0.0, seed: int = 0, offset: int = 0,
                   counter=None, dbias=None, out=None, stream=None):
    """Convenience wrapper over wg_activation_bwd: dx = D(act'(x + bias) dy) in x's type (dy's without x, or `out`, which
    may be x or dy).  dbias (dim,) is written where given, in bias's type."""
    import torch
    xdt = out.dtype if out is not None else x.dtype if x is not None else dy.dtype
    dim = dy.shape[-1]
    b = bias if bias is not None else dbias
    spec = {"tokens": dy.numel() // dim if dim else 0, "dim": dim, "in_dtype": _name(xdt, "dx"), "out_dtype": _name(dy.dtype, "dy"),
            "bias_dtype": "fp32" if b is None else _name(b.dtype, "a bias"),
            **_tail_spec(activation, dropout, seed, offset, counter)}
    nbytes = wg_activation_workspace_size(spec)  # (checks the spec)
    _expect("dy", dy, spec["out_dtype"], dy.shape)
    _expect("x", x, spec["in_dtype"], dy.shape)
    _expect("bias", bias, spec["bias_dtype"], (dim,))
    _expect("dbias", dbias, spec["bias_dtype"], (dim,))
    _expect("out", out, spec["in_dtype"], dy.shape)
    _same_device(dy=dy, x=x, bias=bias, dbias=dbias, out=out, counter=counter)
    with torch.cuda.device(dy.device):
        if out is None:
            out = _empty(stream, dy.shape, xdt, dy.device, returned=True)
        ws = _empty(stream, nbytes, torch.uint8, dy.device) if dbias is not None else None
        wg_activation_bwd(spec, dy, x, out, bias, dbias, ws, None, stream)
    return out
