"""ctypes binding of libselscan (the C ABI declared in include/selscan.h).

Argument marshalling only: every step of the scan runs in the library's CUDA
kernels.  PyTorch supplies device memory (tensors, the cached workspace) and
the current stream.  There is no CPU fallback: if the library is missing or a
call fails, an exception is raised.
"""
import ctypes
import functools
import inspect
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SELSCAN_LIB selects another build of the same library (e.g. one compiled
# with different tuning macros); default: the in-tree build.
LIB_PATH = os.environ.get("SELSCAN_LIB") or os.path.join(_HERE, "csrc", "libselscan.so")

SS_OK = 0
SS_ERR_INVALID_ARG = -1
SS_ERR_UNSUPPORTED = -2
SS_ERR_CUDA = -3
SS_ERR_TIMEOUT = -4
SS_ERR_WORKSPACE = -5

SS_BF16 = 1 << 0
SS_DELTA_SOFTPLUS = 1 << 1
SS_SYNC_CHECK = 1 << 2
SS_FORCE_GENERAL_A = 1 << 3
SS_BETA_SIGMOID = 1 << 4
SS_QK_L2NORM = 1 << 5
SS_TEST_DROP_CARRY = 1 << 30

D_STATE = 16

# Every symbol include/selscan.h declares.
EXPORTED = ("ss_fwd", "ss_step", "ss_fwd_workspace_bytes", "ss_fwd_chunk_len", "ss_check",
            "ss_status_string", "ss_version", "ss_fwd_noalloc", "ss_bwd", "ss_bwd_workspace_bytes",
            "ss_fwd_conv", "ss_step_conv", "ss_block_fwd", "ss_block_scratch_bytes", "ss_ssd_fwd",
            "ss_fwd_host", "ss_fwd_host_workspace_bytes", "ss_ssd_fwd_workspace_bytes", "ss_fwd_with_state",
            "ss_gdr_fwd", "ss_gdr_fwd_workspace_bytes", "ss_gdr_step", "ss_gdr_bwd", "ss_gdr_bwd_workspace_bytes", "ss_norm_fwd", "ss_norm_bwd",
            "ss_norm_bwd_workspace_bytes", "ss_block_fwd_prenorm", "ss_block_prenorm_scratch_bytes")


class ss_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("d_inner", ctypes.c_int64), ("d_state", ctypes.c_int64)]


class ss_launch(ctypes.Structure):
    _fields_ = [("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("timeout_iters", ctypes.c_uint32),
                ("chunk_len", ctypes.c_int32)]


class ss_block_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("in_proj_x", "in_proj_z", "conv_w", "conv_b", "x_proj_dt",
                                                "x_proj_B", "x_proj_C", "dt_proj", "dt_bias", "A", "D",
                                                "out_proj")] + \
               [("d_model", ctypes.c_int64), ("d_inner", ctypes.c_int64), ("dt_rank", ctypes.c_int64)]


BLOCK_WEIGHT_SHAPES = {   # name: (shape as a function of (d_model, d_inner, dt_rank), dtype tag)
    "in_proj_x": (lambda m, i, r: (i, m), "bf16"), "in_proj_z": (lambda m, i, r: (i, m), "bf16"),
    "conv_w": (lambda m, i, r: (i, 4), "f32"), "conv_b": (lambda m, i, r: (i,), "f32"),
    "x_proj_dt": (lambda m, i, r: (r, i), "bf16"), "x_proj_B": (lambda m, i, r: (D_STATE, i), "bf16"),
    "x_proj_C": (lambda m, i, r: (D_STATE, i), "bf16"), "dt_proj": (lambda m, i, r: (i, r), "bf16"),
    "dt_bias": (lambda m, i, r: (i,), "f32"), "A": (lambda m, i, r: (i, D_STATE), "f32"),
    "D": (lambda m, i, r: (i,), "f32"), "out_proj": (lambda m, i, r: (m, i), "bf16"),
}


class ss_ssd_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("d_state", ctypes.c_int64)]


class ss_gdr_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("nheads_k", ctypes.c_int64), ("d_k", ctypes.c_int64), ("d_v", ctypes.c_int64)]


class ss_norm_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class SelscanError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded library with argument types set (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libselscan.so not found at {LIB_PATH}; build it with "
                "`python -m selective_state_space_37_b200.csrc.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, f32p = ctypes.c_void_p, ctypes.c_void_p
        L.ss_fwd.argtypes = [vp, vp, f32p, f32p, vp, vp, f32p, vp, vp, f32p, ctypes.c_uint32,
                             ctypes.POINTER(ss_dims), ctypes.POINTER(ss_launch)]
        L.ss_fwd.restype = ctypes.c_int
        L.ss_step.argtypes = [f32p, vp, vp, f32p, vp, vp, f32p, vp, vp, f32p, ctypes.c_uint32,
                              ctypes.POINTER(ss_dims), ctypes.POINTER(ss_launch)]
        L.ss_step.restype = ctypes.c_int
        L.ss_fwd_workspace_bytes.argtypes = [ctypes.POINTER(ss_dims), ctypes.c_uint32, ctypes.c_int32]
        L.ss_fwd_workspace_bytes.restype = ctypes.c_size_t
        L.ss_fwd_with_state.argtypes = [vp, vp, f32p, f32p, vp, vp, f32p, vp, f32p, vp, f32p, ctypes.c_uint32,
                                        ctypes.POINTER(ss_dims), ctypes.POINTER(ss_launch)]
        L.ss_fwd_with_state.restype = ctypes.c_int
        L.ss_fwd_host.argtypes = [vp, vp, f32p, f32p, vp, vp, f32p, vp, vp, f32p, ctypes.c_uint32,
                                  ctypes.POINTER(ss_dims), ctypes.POINTER(ss_launch), ctypes.c_int32]
        L.ss_fwd_host.restype = ctypes.c_int
        L.ss_fwd_host_workspace_bytes.argtypes = [ctypes.POINTER(ss_dims), ctypes.c_uint32, ctypes.c_int32]
        L.ss_fwd_host_workspace_bytes.restype = ctypes.c_size_t
        L.ss_fwd_chunk_len.argtypes = [ctypes.POINTER(ss_dims), ctypes.c_uint32]
        L.ss_fwd_chunk_len.restype = ctypes.c_int32
        L.ss_check.argtypes = [ctypes.POINTER(ss_launch)]
        L.ss_check.restype = ctypes.c_int
        L.ss_status_string.argtypes = [ctypes.c_int]
        L.ss_status_string.restype = ctypes.c_char_p
        L.ss_version.argtypes = []
        L.ss_version.restype = ctypes.c_int
        L.ss_fwd_noalloc.argtypes = [vp, vp, f32p, f32p, vp, vp, f32p, vp, vp, f32p, ctypes.c_uint32,
                                     ctypes.POINTER(ss_dims), vp]
        L.ss_fwd_noalloc.restype = ctypes.c_int
        L.ss_bwd.argtypes = [vp, vp, f32p, f32p, vp, vp, f32p, vp, vp, f32p, vp, vp, f32p, f32p, f32p,
                             f32p, vp, f32p, ctypes.c_uint32, ctypes.POINTER(ss_dims),
                             ctypes.POINTER(ss_launch)]
        L.ss_bwd.restype = ctypes.c_int
        L.ss_bwd_workspace_bytes.argtypes = [ctypes.POINTER(ss_dims), ctypes.c_uint32]
        L.ss_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ss_fwd_conv.argtypes = [vp, f32p, f32p, vp, f32p, f32p, vp, vp, f32p, vp, vp, f32p, f32p,
                                  ctypes.c_uint32, ctypes.POINTER(ss_dims), ctypes.POINTER(ss_launch)]
        L.ss_fwd_conv.restype = ctypes.c_int
        L.ss_step_conv.argtypes = [f32p, f32p, vp, f32p, f32p, vp, f32p, vp, vp, f32p, vp, vp, f32p,
                                   ctypes.c_uint32, ctypes.POINTER(ss_dims), ctypes.POINTER(ss_launch)]
        L.ss_step_conv.restype = ctypes.c_int
        L.ss_block_fwd.argtypes = [vp, vp, ctypes.POINTER(ss_block_weights), ctypes.c_int64, ctypes.c_int64,
                                   vp, ctypes.c_size_t, vp]
        L.ss_block_fwd.restype = ctypes.c_int
        L.ss_block_scratch_bytes.argtypes = [ctypes.POINTER(ss_block_weights), ctypes.c_int64, ctypes.c_int64]
        L.ss_block_scratch_bytes.restype = ctypes.c_size_t
        L.ss_ssd_fwd.argtypes = [vp, vp, f32p, f32p, vp, vp, f32p, vp, f32p, ctypes.c_uint32,
                                 ctypes.POINTER(ss_ssd_dims), ctypes.POINTER(ss_launch)]
        L.ss_ssd_fwd.restype = ctypes.c_int
        L.ss_ssd_fwd_workspace_bytes.argtypes = [ctypes.POINTER(ss_ssd_dims), ctypes.c_uint32]
        L.ss_ssd_fwd_workspace_bytes.restype = ctypes.c_size_t
        gp, np_ = ctypes.POINTER(ss_gdr_dims), ctypes.POINTER(ss_norm_dims)
        u32, f32, lp = ctypes.c_uint32, ctypes.c_float, ctypes.POINTER(ss_launch)
        L.ss_gdr_fwd.argtypes = [vp, vp, vp, vp, f32p, f32p, vp, f32p, vp, vp, f32p, f32, u32, gp, lp]
        L.ss_gdr_step.argtypes = [f32p, vp, vp, vp, vp, f32p, f32p, vp, vp, f32, u32, gp, lp]
        L.ss_gdr_bwd.argtypes = [vp] * 19 + [f32, u32, gp, lp]
        L.ss_norm_fwd.argtypes = [vp, f32p, f32p, vp, f32p, f32p, f32, u32, np_, lp]
        L.ss_norm_bwd.argtypes = [vp, vp, f32p, f32p, f32p, vp, f32p, f32p, u32, np_, lp]
        L.ss_block_fwd_prenorm.argtypes = [vp, f32p, f32p, f32, vp, ctypes.POINTER(ss_block_weights),
                                           ctypes.c_int64, ctypes.c_int64, vp, ctypes.c_size_t, vp]
        for f in (L.ss_gdr_fwd, L.ss_gdr_step, L.ss_gdr_bwd, L.ss_norm_fwd, L.ss_norm_bwd, L.ss_block_fwd_prenorm):
            f.restype = ctypes.c_int
        L.ss_gdr_fwd_workspace_bytes.argtypes = [gp, u32, ctypes.c_int32]
        L.ss_norm_bwd_workspace_bytes.argtypes = [np_, u32]
        L.ss_block_prenorm_scratch_bytes.argtypes = [ctypes.POINTER(ss_block_weights), ctypes.c_int64,
                                                     ctypes.c_int64]
        L.ss_gdr_bwd_workspace_bytes.argtypes = [gp, u32]
        for f in (L.ss_gdr_fwd_workspace_bytes, L.ss_gdr_bwd_workspace_bytes, L.ss_norm_bwd_workspace_bytes, L.ss_block_prenorm_scratch_bytes):
            f.restype = ctypes.c_size_t
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ss_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else t.data_ptr()   # (a c_void_p argument takes the number)


def _io_flag(t):
    if t.dtype == torch.bfloat16:
        return SS_BF16
    if t.dtype == torch.float32:
        return 0
    raise TypeError(f"u/delta/z/B/C must be bfloat16 or float32, got {t.dtype}")


def _check(t, name, shape, dtype, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return   # (small calls spend more time here than on the GPU)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_ws_cache = {}


def workspace_for(nbytes, device, stream_handle):
    """A cached device workspace of at least nbytes for (device, stream).

    One buffer per (device, stream), grown when a call needs more; calls on
    one stream run in order (_in_turn keeps host threads' launches apart), so
    they can share it.  A replaced buffer is returned to torch's
    stream-ordered allocator.  clear_workspaces() drops them all."""
    key = (device.index, int(stream_handle))
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


_ws_locks = {}


def _in_turn(device, stream_handle):
    """The lock of a (device, stream), held from a call's look-up of the cached workspace to its last launch: a call
    is several launches on one workspace, and ctypes lets other threads run between them."""
    key = (device.index, stream_handle)
    return _ws_locks.get(key) or _ws_locks.setdefault(key, threading.RLock())


def clear_workspaces():
    """Releases the cached workspaces (call after synchronizing the streams
    that used them)."""
    _ws_cache.clear()


def _stream_handle(stream, device):
    if stream is None:
        index = torch.cuda.current_device() if device.index is None else device.index
        return torch._C._cuda_getCurrentRawStream(index)   # torch.cuda.current_stream() without its object
    return stream.cuda_stream


def _on_stream(fn):
    """Runs a function with the stream that it is given as the current one: what it makes -- outputs, the cached
    workspace -- is that stream's then.  (The allocator may hand out a block of the current stream's that work queued there
    still uses, and hands a freed one out again behind the work of its own stream.)"""
    @functools.wraps(fn)
    def call(*args, **kw):
        stream = kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _on_device(fn):
    """Runs a function with its first tensor's device current (the library launches on the current device)."""
    name = inspect.unwrap(fn).__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, **kw):
        dev = getattr(args[0] if args else kw.get(name), "device", None)
        if dev is None or dev.type != "cuda":
            raise ValueError(f"{fn.__name__} runs on CUDA tensors only ({name})")
        if dev.index == torch.cuda.current_device():
            return fn(*args, **kw)
        with torch.cuda.device(dev):
            return fn(*args, **kw)
    return call


def _launch_for(need, dev, sh, workspace, timeout_iters=0, chunk_len=0):
    """(the call's ss_launch, its workspace): the tensor is the caller's to hold until the library has returned, since
    the cache may let go of it before (another thread's larger request on the same stream)."""
    if workspace is None:
        # a captured graph gets a workspace of its own, from its memory pool: graphs may be replayed at once,
        # and the cached buffer may have been replaced by a larger one by then
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev) if \
            torch.cuda.is_current_stream_capturing() else workspace_for(need, dev, sh)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return ss_launch(sh, workspace.data_ptr(), workspace.numel() * workspace.element_size(), int(timeout_iters),
                     int(chunk_len)), workspace


def fwd_workspace_bytes(batch, seqlen, d_inner, bf16=True, chunk_len=0, d_state=D_STATE):
    dims = ss_dims(batch, seqlen, d_inner, d_state)
    return int(lib().ss_fwd_workspace_bytes(ctypes.byref(dims), SS_BF16 if bf16 else 0, int(chunk_len)))


def fwd_chunk_len(batch, seqlen, d_inner, bf16=True, d_state=D_STATE):
    dims = ss_dims(batch, seqlen, d_inner, d_state)
    return int(lib().ss_fwd_chunk_len(ctypes.byref(dims), SS_BF16 if bf16 else 0))


@_on_stream
def ss_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, y=None, last_state=None,
           return_last_state=True, softplus=True, force_general_A=False, chunk_len=0,
           timeout_iters=0, workspace=None, stream=None, sync_check=False, extra_flags=0,
           initial_state=None):
    """Selective-scan forward pass through libselscan's ss_fwd (or
    ss_fwd_with_state when initial_state [batch, d_inner, 16] fp32 is given).

    u, delta, z: [batch, L, d_inner]; B, C: [batch, L, 16] (bf16 or fp32, all the
    same); A: [d_inner, 16] fp32; D, delta_bias: [d_inner] fp32 or None.
    Returns (y, last_state); last_state is None when return_last_state is False
    and none was passed in.
    """
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, d_inner]")
    batch, L, d = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("ss_fwd runs on CUDA tensors only")
    io = u.dtype
    for t, nm, shp in ((u, "u", (batch, L, d)), (delta, "delta", (batch, L, d)),
                       (z, "z", (batch, L, d)), (B, "B", (batch, L, D_STATE)),
                       (C, "C", (batch, L, D_STATE))):
        _check(t, nm, shp, io, dev)
    _check(A, "A", (d, D_STATE), torch.float32, dev)
    _check(D, "D", (d,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (d,), torch.float32, dev)
    if y is None:
        y = torch.empty((batch, L, d), dtype=io, device=dev)
    _check(y, "y", (batch, L, d), io, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, d, D_STATE), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, d, D_STATE), torch.float32, dev)
    flags = _io_flag(u) | (SS_DELTA_SOFTPLUS if softplus else 0) | int(extra_flags)
    if force_general_A:
        flags |= SS_FORCE_GENERAL_A
    if sync_check:
        flags |= SS_SYNC_CHECK
    dims = ss_dims(batch, L, d, D_STATE)
    need = int(lib().ss_fwd_workspace_bytes(ctypes.byref(dims), flags, int(chunk_len)))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace, timeout_iters, chunk_len)
        if initial_state is not None:
            _check(initial_state, "initial_state", (batch, d, D_STATE), torch.float32, dev)
            rc = lib().ss_fwd_with_state(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                         _ptr(z), _ptr(initial_state), _ptr(y), _ptr(last_state), flags,
                                         ctypes.byref(dims), ctypes.byref(launch))
        else:
            rc = lib().ss_fwd(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                              _ptr(z), _ptr(y), _ptr(last_state), flags, ctypes.byref(dims),
                              ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_fwd")
    return y, last_state


@_on_stream
def ss_fwd_host(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, y=None, last_state=None,
                return_last_state=True, softplus=True, rows_per_slice=1, workspace=None, stream=None,
                sync_check=False):
    """ss_fwd on activations in host memory through libselscan's ss_fwd_host.

    u, delta, z, B, C (and y, last_state if given) are CPU tensors -- pinned
    for overlapped copies -- with ss_fwd's shapes; A, D, delta_bias are CUDA
    tensors on the device that runs the scan.  Batch slices of rows_per_slice
    rows are uploaded, scanned and downloaded with the three overlapped.
    Returns (y, last_state) as CPU tensors, complete once the stream is
    synchronized (sync_check=True does it).
    """
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, d_inner]")
    batch, L, d = u.shape
    host = torch.device("cpu")
    dev = A.device
    if dev.type != "cuda":
        raise ValueError("A, D and delta_bias must be CUDA tensors")
    io = u.dtype
    for t, nm, shp in ((u, "u", (batch, L, d)), (delta, "delta", (batch, L, d)),
                       (z, "z", (batch, L, d)), (B, "B", (batch, L, D_STATE)),
                       (C, "C", (batch, L, D_STATE))):
        _check(t, nm, shp, io, host)
    _check(A, "A", (d, D_STATE), torch.float32, dev)
    _check(D, "D", (d,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (d,), torch.float32, dev)
    pin = u.is_pinned()
    if y is None:
        y = torch.empty((batch, L, d), dtype=io, pin_memory=pin)
    _check(y, "y", (batch, L, d), io, host)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, d, D_STATE), dtype=torch.float32, pin_memory=pin)
    _check(last_state, "last_state", (batch, d, D_STATE), torch.float32, host)
    flags = _io_flag(u) | (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_SYNC_CHECK if sync_check else 0)
    dims = ss_dims(batch, L, d, D_STATE)
    need = int(lib().ss_fwd_host_workspace_bytes(ctypes.byref(dims), flags, int(rows_per_slice)))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace)
        rc = lib().ss_fwd_host(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                               _ptr(z), _ptr(y), _ptr(last_state), flags, ctypes.byref(dims),
                               ctypes.byref(launch), int(rows_per_slice))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_fwd_host")
    return y, last_state


def fwd_host_workspace_bytes(batch, seqlen, d_inner, bf16=True, rows_per_slice=1, d_state=D_STATE):
    dims = ss_dims(batch, seqlen, d_inner, d_state)
    return int(lib().ss_fwd_host_workspace_bytes(ctypes.byref(dims), SS_BF16 if bf16 else 0, int(rows_per_slice)))


def bwd_workspace_bytes(batch, seqlen, d_inner, bf16=True, d_state=D_STATE):
    dims = ss_dims(batch, seqlen, d_inner, d_state)
    return int(lib().ss_bwd_workspace_bytes(ctypes.byref(dims), SS_BF16 if bf16 else 0))


@_on_stream
def ss_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, dlast_state=None, *,
           softplus=True, grads=None, chunk_len=0, workspace=None, stream=None, sync_check=False):
    """Backward of ss_fwd through libselscan's ss_bwd.

    Same inputs as ss_fwd plus dy [batch, L, d_inner] (the element type of u)
    and dlast_state [batch, d_inner, 16] fp32 or None.  Returns a dict with
    du, ddelta, dz (element type of u; dz only with z), dA [d_inner, 16],
    dB, dC [batch, L, 16], dD and ddelta_bias [d_inner] (fp32; only with D /
    delta_bias).  `grads` may supply preallocated output tensors by name;
    chunk_len > 0 fixes the time-chunk length (0: the library's choice).
    """
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, d_inner]")
    batch, L, d = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("ss_bwd runs on CUDA tensors only")
    io = u.dtype
    for t, nm, shp in ((u, "u", (batch, L, d)), (delta, "delta", (batch, L, d)),
                       (z, "z", (batch, L, d)), (dy, "dy", (batch, L, d)),
                       (B, "B", (batch, L, D_STATE)), (C, "C", (batch, L, D_STATE))):
        _check(t, nm, shp, io, dev)
    _check(A, "A", (d, D_STATE), torch.float32, dev)
    _check(D, "D", (d,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (d,), torch.float32, dev)
    _check(dlast_state, "dlast_state", (batch, d, D_STATE), torch.float32, dev)
    g = dict(grads or {})
    shapes = {"du": ((batch, L, d), io), "ddelta": ((batch, L, d), io), "dA": ((d, D_STATE), torch.float32),
              "dB": ((batch, L, D_STATE), torch.float32), "dC": ((batch, L, D_STATE), torch.float32)}
    if z is not None:
        shapes["dz"] = ((batch, L, d), io)
    if D is not None:
        shapes["dD"] = ((d,), torch.float32)
    if delta_bias is not None:
        shapes["ddelta_bias"] = ((d,), torch.float32)
    for k, (shp, dt) in shapes.items():
        if k not in g:
            g[k] = torch.empty(shp, dtype=dt, device=dev)
        _check(g[k], k, shp, dt, dev)
    flags = _io_flag(u) | (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_SYNC_CHECK if sync_check else 0)
    dims = ss_dims(batch, L, d, D_STATE)
    need = int(lib().ss_bwd_workspace_bytes(ctypes.byref(dims), flags))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace, 0, chunk_len)
        rc = lib().ss_bwd(_ptr(u), _ptr(delta), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                          _ptr(dy), _ptr(dlast_state), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]),
                          _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g.get("dD")), _ptr(g.get("dz")),
                          _ptr(g.get("ddelta_bias")), flags, ctypes.byref(dims), ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_bwd")
    return {k: g[k] for k in shapes}


@_on_stream
def ss_fwd_conv(x, conv_w, delta, A, B, C, D=None, z=None, delta_bias=None, conv_b=None, *, y=None,
                last_state=None, return_last_state=True, conv_state=None, softplus=True, chunk_len=0,
                timeout_iters=0, workspace=None, stream=None, sync_check=False):
    """ss_fwd with the causal conv1d (width 4) + SiLU prologue: x takes u's
    place, conv_w [d_inner, 4] fp32, conv_b [d_inner] fp32 or None.  Returns
    (y, last_state); pass conv_state [batch, d_inner, 3] fp32 to receive the
    last three x of each channel (for ss_step_conv)."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, d_inner]")
    batch, L, d = x.shape
    dev = x.device
    io = x.dtype
    for t, nm, shp in ((x, "x", (batch, L, d)), (delta, "delta", (batch, L, d)),
                       (z, "z", (batch, L, d)), (B, "B", (batch, L, D_STATE)),
                       (C, "C", (batch, L, D_STATE))):
        _check(t, nm, shp, io, dev)
    _check(conv_w, "conv_w", (d, 4), torch.float32, dev)
    _check(conv_b, "conv_b", (d,), torch.float32, dev)
    _check(A, "A", (d, D_STATE), torch.float32, dev)
    _check(D, "D", (d,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (d,), torch.float32, dev)
    _check(conv_state, "conv_state", (batch, d, 3), torch.float32, dev)
    if y is None:
        y = torch.empty((batch, L, d), dtype=io, device=dev)
    _check(y, "y", (batch, L, d), io, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, d, D_STATE), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, d, D_STATE), torch.float32, dev)
    flags = _io_flag(x) | (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_SYNC_CHECK if sync_check else 0)
    dims = ss_dims(batch, L, d, D_STATE)
    need = int(lib().ss_fwd_workspace_bytes(ctypes.byref(dims), flags, int(chunk_len)))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace, timeout_iters, chunk_len)
        rc = lib().ss_fwd_conv(_ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(delta), _ptr(delta_bias), _ptr(A),
                               _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(last_state), _ptr(conv_state),
                               flags, ctypes.byref(dims), ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_fwd_conv")
    return y, last_state


@_on_stream
def ss_step_conv(state, conv_state, x, conv_w, delta, A, B, C, D=None, z=None, delta_bias=None, conv_b=None,
                 *, y=None, softplus=True, stream=None, sync_check=False):
    """One decode step with the conv prologue; state [batch, d_inner, 16] and
    conv_state [batch, d_inner, 3] (fp32) are updated in place.  Returns y."""
    batch, d = x.shape
    dev = x.device
    io = x.dtype
    _check(state, "state", (batch, d, D_STATE), torch.float32, dev)
    _check(conv_state, "conv_state", (batch, d, 3), torch.float32, dev)
    for t, nm, shp in ((x, "x", (batch, d)), (delta, "delta", (batch, d)), (z, "z", (batch, d)),
                       (B, "B", (batch, D_STATE)), (C, "C", (batch, D_STATE))):
        _check(t, nm, shp, io, dev)
    _check(conv_w, "conv_w", (d, 4), torch.float32, dev)
    _check(conv_b, "conv_b", (d,), torch.float32, dev)
    _check(A, "A", (d, D_STATE), torch.float32, dev)
    _check(D, "D", (d,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (d,), torch.float32, dev)
    if y is None:
        y = torch.empty((batch, d), dtype=io, device=dev)
    flags = _io_flag(x) | (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_SYNC_CHECK if sync_check else 0)
    sh = _stream_handle(stream, dev)
    dims = ss_dims(batch, 1, d, D_STATE)
    launch = ss_launch(sh, None, 0, 0, 0)
    rc = lib().ss_step_conv(_ptr(state), _ptr(conv_state), _ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(delta),
                            _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(delta_bias), flags,
                            ctypes.byref(dims), ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_step_conv")
    return y


def _block_struct(weights, device):
    d_inner, d_model = weights["in_proj_x"].shape
    dt_rank = weights["x_proj_dt"].shape[0]
    st = ss_block_weights()
    for name, (shape_fn, tag) in BLOCK_WEIGHT_SHAPES.items():
        t = weights.get(name)
        if t is None and name in ("conv_b", "D"):
            continue
        _check(t, name, shape_fn(d_model, d_inner, dt_rank), torch.bfloat16 if tag == "bf16" else torch.float32,
               device)
        setattr(st, name, t.data_ptr())
    st.d_model, st.d_inner, st.dt_rank = d_model, d_inner, dt_rank
    return st


def block_scratch_bytes(weights, batch, seqlen):
    st = _block_struct(weights, weights["in_proj_x"].device)
    return int(lib().ss_block_scratch_bytes(ctypes.byref(st), batch, seqlen))


@_on_stream
def ss_block_fwd(hidden, weights, *, out=None, scratch=None, stream=None):
    """Forward of one Mamba block's inner path through libselscan's
    ss_block_fwd.  hidden [batch, L, d_model] bf16; weights: a dict of
    tensors named as the fields of ss_block_weights (bf16 matrices, fp32
    vectors).  Returns out [batch, L, d_model] bf16."""
    batch, L, d_model = hidden.shape
    dev = hidden.device
    st = _block_struct(weights, dev)
    if st.d_model != d_model:
        raise ValueError("hidden's last dimension must equal d_model")
    _check(hidden, "hidden", (batch, L, d_model), torch.bfloat16, dev)
    if out is None:
        out = torch.empty_like(hidden)
    _check(out, "out", (batch, L, d_model), torch.bfloat16, dev)
    need = int(lib().ss_block_scratch_bytes(ctypes.byref(st), batch, L))
    if need == 0:
        raise SelscanError(SS_ERR_INVALID_ARG, "ss_block_fwd")
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, scratch = _launch_for(need, dev, sh, scratch)
        rc = lib().ss_block_fwd(_ptr(hidden), _ptr(out), ctypes.byref(st), batch, L, launch.workspace,
                                launch.workspace_bytes, launch.stream)
    if rc != SS_OK:
        raise SelscanError(rc, "ss_block_fwd")
    return out


@_on_stream
def ss_ssd_fwd(x, dt, A, B, C, D=None, dt_bias=None, *, softplus=True, y=None, final_state=None,
               return_final_state=True, chunk_len=0, split=True, workspace=None, stream=None, sync_check=False,
               timeout_iters=0, extra_flags=0):
    """Multi-head scan with a scalar decay per head (Mamba-2's SSD model).
    x [batch, L, nheads, 64] bf16; dt [batch, L, nheads] bf16; A [nheads] fp32;
    B, C [batch, L, d_state] bf16 (d_state 64 or 128); D, dt_bias [nheads] fp32
    or None.  Returns (y [batch, L, nheads, 64] bf16, final_state
    [batch, nheads, 64, d_state] fp32 or None).  split=False runs every
    sequence whole (no workspace); chunk_len > 0 fixes the segment length;
    timeout_iters bounds one wait in microseconds (0: two
    seconds); extra_flags adds raw SS_* flags (SS_TEST_DROP_CARRY in tests)."""
    batch, L, H, P = x.shape
    N = B.shape[-1]
    dev = x.device
    bf = torch.bfloat16
    _check(x, "x", (batch, L, H, P), bf, dev)
    _check(dt, "dt", (batch, L, H), bf, dev)
    _check(B, "B", (batch, L, N), bf, dev)
    _check(C, "C", (batch, L, N), bf, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(D, "D", (H,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    _check(y, "y", (batch, L, H, P), bf, dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, H, P, N), dtype=torch.float32, device=dev)
    _check(final_state, "final_state", (batch, H, P, N), torch.float32, dev)
    flags = (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_SYNC_CHECK if sync_check else 0) | int(extra_flags)
    dims = ss_ssd_dims(batch, L, H, P, N)
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        if split:
            need = int(lib().ss_ssd_fwd_workspace_bytes(ctypes.byref(dims), flags))
            launch, workspace = _launch_for(need, dev, sh, workspace, timeout_iters, chunk_len)
        else:
            launch = ss_launch(sh, None, 0, int(timeout_iters), int(chunk_len))
        rc = lib().ss_ssd_fwd(_ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(y),
                              _ptr(final_state), flags, ctypes.byref(dims), ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_ssd_fwd")
    return y, final_state


def _gdr_setup(q, k, v, dt, A, beta, dt_bias, io, softplus, beta_sigmoid, qk_l2norm, tok):
    """Checks the inputs that the ss_gdr_* calls share (`tok`: the token dimensions, [batch] or
    [batch, L]) and returns (dims, flags)."""
    n = len(tok)
    for t, name in ((q, "q"), (v, "v")):
        if t.dim() != n + 2:
            raise ValueError(f"{name} must have {n + 2} dimensions")
    hk, d_k = q.shape[n:]
    h, d_v = v.shape[n:]
    dev = q.device
    for t, name, shape in ((q, "q", (*tok, hk, d_k)), (k, "k", (*tok, hk, d_k)), (v, "v", (*tok, h, d_v)),
                           (dt, "dt", (*tok, h)), (beta, "beta", (*tok, h))):
        _check(t, name, shape, io, dev)
    _check(A, "A", (h,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (h,), torch.float32, dev)
    flags = _io_flag(q) | (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_BETA_SIGMOID if beta_sigmoid else 0) | \
        (SS_QK_L2NORM if qk_l2norm else 0)
    return ss_gdr_dims(tok[0], tok[1] if n > 1 else 1, h, hk, d_k, d_v), flags


@_on_device
@_on_stream
def ss_gdr_fwd(q, k, v, dt, A, beta, dt_bias=None, initial_state=None, seqlens=None, *, scale=None, softplus=True,
               beta_sigmoid=True, qk_l2norm=True, y=None, final_state=None, return_final_state=True, chunk_len=0,
               workspace=None, stream=None, sync_check=False, timeout_iters=0, extra_flags=0):
    """Gated delta rule over a sequence through libselscan's ss_gdr_fwd.
    q, k [batch, L, nheads_k, d_k]; v [batch, L, nheads, d_v]; dt, beta [batch, L, nheads] (bf16 or fp32,
    all the same; d_k, d_v 64 or 128; nheads a multiple of nheads_k); A, dt_bias [nheads] fp32;
    initial_state [batch, nheads, d_v, d_k] fp32 or None; seqlens [batch] int32 on the device or None:
    the tokens of each sequence, the rows of y behind them staying as they were (zero when y is made
    here).  With stream=, outputs that the call makes are that stream's.  scale defaults to d_k ** -0.5.
    Returns (y, final_state or None); final_state may be initial_state."""
    if q.dim() != 4:
        raise ValueError("q must be [batch, L, nheads_k, d_k]")
    batch, L = q.shape[:2]
    dims, flags = _gdr_setup(q, k, v, dt, A, beta, dt_bias, q.dtype, softplus, beta_sigmoid, qk_l2norm, (batch, L))
    dev = q.device
    states = (batch, dims.nheads, dims.d_v, dims.d_k)
    _check(initial_state, "initial_state", states, torch.float32, dev)
    _check(seqlens, "seqlens", (batch,), torch.int32, dev)
    if y is None:
        y = torch.empty_like(v)
        if seqlens is not None:
            y.zero_()
    _check(y, "y", v.shape, v.dtype, dev)
    if final_state is None and return_final_state:
        final_state = torch.empty(states, dtype=torch.float32, device=dev)
    _check(final_state, "final_state", states, torch.float32, dev)
    flags |= (SS_SYNC_CHECK if sync_check else 0) | int(extra_flags)
    need = int(lib().ss_gdr_fwd_workspace_bytes(ctypes.byref(dims), flags, int(chunk_len)))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace, timeout_iters, chunk_len)
        rc = lib().ss_gdr_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(beta),
                              _ptr(initial_state), _ptr(seqlens), _ptr(y), _ptr(final_state),
                              dims.d_k ** -0.5 if scale is None else float(scale), flags, ctypes.byref(dims),
                              ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_gdr_fwd")
    return y, final_state


@_on_device
@_on_stream
def ss_gdr_step(state, q, k, v, dt, A, beta, dt_bias=None, *, scale=None, softplus=True, beta_sigmoid=True,
                qk_l2norm=True, y=None, stream=None, sync_check=False):
    """One token of the gated delta rule through libselscan's ss_gdr_step; `state`
    [batch, nheads, d_v, d_k] fp32 is updated in place.  q, k [batch, nheads_k, d_k]; v [batch, nheads, d_v];
    dt, beta [batch, nheads]; the rest as in ss_gdr_fwd.  Returns y [batch, nheads, d_v]."""
    if state.dim() != 4:
        raise ValueError("state must be [batch, nheads, d_v, d_k]")
    dev = state.device
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, expected {dev}")
    dims, flags = _gdr_setup(q, k, v, dt, A, beta, dt_bias, q.dtype, softplus, beta_sigmoid, qk_l2norm,
                             (state.shape[0],))
    _check(state, "state", (dims.batch, dims.nheads, dims.d_v, dims.d_k), torch.float32, dev)
    if y is None:
        y = torch.empty_like(v)
    _check(y, "y", v.shape, v.dtype, dev)
    flags |= SS_SYNC_CHECK if sync_check else 0
    launch = ss_launch(_stream_handle(stream, dev), None, 0, 0, 0)
    rc = lib().ss_gdr_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(beta),
                           _ptr(y), dims.d_k ** -0.5 if scale is None else float(scale), flags, ctypes.byref(dims),
                           ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_gdr_step")
    return y


@_on_device
@_on_stream
def ss_gdr_bwd(q, k, v, dt, A, beta, dy, dt_bias=None, initial_state=None, dfinal_state=None, seqlens=None, *,
               scale=None, softplus=True, beta_sigmoid=True, qk_l2norm=True, grads=None, workspace=None, stream=None,
               sync_check=False, timeout_iters=0, extra_flags=0):
    """Backward of ss_gdr_fwd through libselscan's ss_gdr_bwd.  Its inputs, dy like v and dfinal_state
    [batch, nheads, d_v, d_k] fp32 or None.  Returns a dict with dq, dk, dv, ddt, dbeta (of the type and shape
    of what they are of), dA, ddt_bias (fp32; the latter with dt_bias) and dinitial_state (fp32, with
    initial_state); `grads` may supply output tensors by name."""
    if q.dim() != 4:
        raise ValueError("q must be [batch, L, nheads_k, d_k]")
    batch, L = q.shape[:2]
    dims, flags = _gdr_setup(q, k, v, dt, A, beta, dt_bias, q.dtype, softplus, beta_sigmoid, qk_l2norm, (batch, L))
    dev = q.device
    states = (batch, dims.nheads, dims.d_v, dims.d_k)
    _check(dy, "dy", v.shape, v.dtype, dev)
    _check(initial_state, "initial_state", states, torch.float32, dev)
    _check(dfinal_state, "dfinal_state", states, torch.float32, dev)
    _check(seqlens, "seqlens", (batch,), torch.int32, dev)
    like = {"dq": q, "dk": k, "dv": v, "ddt": dt, "dbeta": beta, "dA": A}
    if dt_bias is not None:
        like["ddt_bias"] = dt_bias
    if initial_state is not None:
        like["dinitial_state"] = initial_state
    if grads and not like.keys() >= grads.keys():
        raise ValueError(f"grads: no {sorted(grads.keys() - like.keys())} in this call's gradients {sorted(like)}")
    g = {}
    for name, t in like.items():
        given = (grads or {}).get(name)
        g[name] = torch.empty_like(t) if given is None else given
        _check(g[name], name, t.shape, t.dtype, dev)
    flags |= (SS_SYNC_CHECK if sync_check else 0) | int(extra_flags)
    need = int(lib().ss_gdr_bwd_workspace_bytes(ctypes.byref(dims), flags))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace, timeout_iters)
        rc = lib().ss_gdr_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(beta),
                              _ptr(initial_state), _ptr(seqlens), _ptr(dy), _ptr(dfinal_state), _ptr(g["dq"]),
                              _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["ddt"]), _ptr(g["dbeta"]), _ptr(g["dA"]),
                              _ptr(g.get("ddt_bias")), _ptr(g.get("dinitial_state")),
                              dims.d_k ** -0.5 if scale is None else float(scale), flags, ctypes.byref(dims),
                              ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_gdr_bwd")
    return g


@_on_device
@_on_stream
def ss_norm_fwd(x, weight=None, bias=None, *, eps=1e-5, y=None, stats=True, stream=None, sync_check=False):
    """Layer norm over the last dimension of x (bf16 or fp32, contiguous) through libselscan's
    ss_norm_fwd; weight, bias [cols] fp32 or None; y may be x.  Returns (y, mean, rstd), the statistics
    [rows] in fp32 for ss_norm_bwd (None with stats=False)."""
    if x.dim() == 0:
        raise ValueError("x needs at least one dimension")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    dev = x.device
    _check(x, "x", x.shape, x.dtype, dev)
    _check(weight, "weight", (cols,), torch.float32, dev)
    _check(bias, "bias", (cols,), torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    _check(y, "y", x.shape, x.dtype, dev)
    mean = torch.empty(rows, dtype=torch.float32, device=dev) if stats else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if stats else None
    flags = _io_flag(x) | (SS_SYNC_CHECK if sync_check else 0)
    dims = ss_norm_dims(rows, cols)
    launch = ss_launch(_stream_handle(stream, dev), None, 0, 0, 0)
    rc = lib().ss_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), float(eps), flags,
                           ctypes.byref(dims), ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_norm_fwd")
    return y, mean, rstd


@_on_device
@_on_stream
def ss_norm_bwd(dy, x, mean, rstd, weight=None, *, dx=None, dweight=None, dbias=None, sums=True, workspace=None,
                stream=None, sync_check=False):
    """Backward of ss_norm_fwd through libselscan's ss_norm_bwd: dy and x of one shape and type, mean and
    rstd [rows] fp32 from the forward, weight [cols] fp32 or None; dx may be dy.  Returns a dict with
    dx, dweight and dbias (fp32 [cols]; without them for sums=False)."""
    if x.dim() == 0:
        raise ValueError("x needs at least one dimension")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    dev = dy.device
    _check(x, "x", x.shape, x.dtype, dev)
    _check(dy, "dy", x.shape, x.dtype, dev)
    _check(mean, "mean", (rows,), torch.float32, dev)
    _check(rstd, "rstd", (rows,), torch.float32, dev)
    _check(weight, "weight", (cols,), torch.float32, dev)
    g = {"dx": torch.empty_like(x) if dx is None else dx}
    _check(g["dx"], "dx", x.shape, x.dtype, dev)
    if sums:
        for name, t in (("dweight", dweight), ("dbias", dbias)):
            g[name] = torch.empty(cols, dtype=torch.float32, device=dev) if t is None else t
            _check(g[name], name, (cols,), torch.float32, dev)
    flags = _io_flag(x) | (SS_SYNC_CHECK if sync_check else 0)
    dims = ss_norm_dims(rows, cols)
    need = int(lib().ss_norm_bwd_workspace_bytes(ctypes.byref(dims), flags))
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, workspace = _launch_for(need, dev, sh, workspace)
        rc = lib().ss_norm_bwd(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(g["dx"]),
                               _ptr(g.get("dweight")), _ptr(g.get("dbias")), flags, ctypes.byref(dims),
                               ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_norm_bwd")
    return g


@_on_device
@_on_stream
def ss_block_fwd_prenorm(hidden, weights, norm_weight=None, norm_bias=None, *, eps=1e-5, out=None, scratch=None,
                         stream=None):
    """hidden + block(layer_norm(hidden)) through libselscan's ss_block_fwd_prenorm: ss_block_fwd's arguments,
    norm_weight and norm_bias [d_model] fp32 or None.  out must not be hidden."""
    if hidden.dim() != 3:
        raise ValueError("hidden must be [batch, L, d_model]")
    batch, L, d_model = hidden.shape
    dev = hidden.device
    st = _block_struct(weights, dev)
    if st.d_model != d_model:
        raise ValueError("hidden's last dimension must equal d_model")
    _check(hidden, "hidden", (batch, L, d_model), torch.bfloat16, dev)
    _check(norm_weight, "norm_weight", (d_model,), torch.float32, dev)
    _check(norm_bias, "norm_bias", (d_model,), torch.float32, dev)
    if out is None:
        out = torch.empty_like(hidden)
    _check(out, "out", (batch, L, d_model), torch.bfloat16, dev)
    need = int(lib().ss_block_prenorm_scratch_bytes(ctypes.byref(st), batch, L))
    if need == 0:
        raise SelscanError(SS_ERR_INVALID_ARG, "ss_block_fwd_prenorm")
    sh = _stream_handle(stream, dev)
    with _in_turn(dev, sh):
        launch, scratch = _launch_for(need, dev, sh, scratch)
        rc = lib().ss_block_fwd_prenorm(_ptr(hidden), _ptr(norm_weight), _ptr(norm_bias), float(eps), _ptr(out),
                                        ctypes.byref(st), batch, L, launch.workspace, launch.workspace_bytes,
                                        launch.stream)
    if rc != SS_OK:
        raise SelscanError(rc, "ss_block_fwd_prenorm")
    return out


def ss_check(workspace, stream=None, device=None):
    """Synchronize and return the device status recorded in `workspace`."""
    dev = workspace.device if device is None else device
    sh = _stream_handle(stream, dev)
    launch = ss_launch(sh, workspace.data_ptr(), workspace.numel() * workspace.element_size(), 0, 0)
    return int(lib().ss_check(ctypes.byref(launch)))


@_on_stream
def ss_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, y=None, softplus=True,
            stream=None, sync_check=False):
    """One decode step through libselscan's ss_step; `state` is updated in place.

    state: [batch, d_inner, 16] fp32; u, delta, z: [batch, d_inner]; B, C: [batch, 16]
    (bf16 or fp32); A: [d_inner, 16] fp32; D, delta_bias: [d_inner] fp32 or None.
    Returns y [batch, d_inner].
    """
    if state.dim() != 3:
        raise ValueError("state must be [batch, d_inner, 16]")
    batch, d, _ = state.shape
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("ss_step runs on CUDA tensors only")
    io = u.dtype
    _check(state, "state", (batch, d, D_STATE), torch.float32, dev)
    for t, nm, shp in ((u, "u", (batch, d)), (delta, "delta", (batch, d)), (z, "z", (batch, d)),
                       (B, "B", (batch, D_STATE)), (C, "C", (batch, D_STATE))):
        _check(t, nm, shp, io, dev)
    _check(A, "A", (d, D_STATE), torch.float32, dev)
    _check(D, "D", (d,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (d,), torch.float32, dev)
    if y is None:
        y = torch.empty((batch, d), dtype=io, device=dev)
    _check(y, "y", (batch, d), io, dev)
    flags = _io_flag(u) | (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_SYNC_CHECK if sync_check else 0)
    sh = _stream_handle(stream, dev)
    dims = ss_dims(batch, 1, d, D_STATE)
    launch = ss_launch(sh, None, 0, 0, 0)
    rc = lib().ss_step(_ptr(state), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                       _ptr(z), _ptr(y), _ptr(delta_bias), flags, ctypes.byref(dims),
                       ctypes.byref(launch))
    if rc != SS_OK:
        raise SelscanError(rc, "ss_step")
    return y
