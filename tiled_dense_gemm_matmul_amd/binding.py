"""Python binding over libgemmfwd.so (the C ABI declared in include/*.h).

Argument marshalling only: shapes, dtypes and devices are checked, pointers and
the current HIP stream are passed through, and every step of the computation
runs in the library's HIP kernels.  torch provides device memory and streams.
The library must be built (``__graft_entry__.build()``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

GEMM_FLAG_W_F16 = 0x1
GEMM_FLAG_ACC = 0x2
GEMM_W_F32 = 0
GEMM_W_F16 = 1

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgemmfwd.so")
_lib = None

EXPORTED = (
    "gemm_fwd", "gemm_fwd_swiglu", "gemm_fwd_ex", "gemm_fwd_swiglu_ex", "gemm_fwd_workspace_bytes",
    "gemm_fwd_swiglu_noalloc",
    "gemm_num_configs", "gemm_config_name", "gemm_select_config", "gemm_status_string",
    "gemm_matmul_t", "gemm_matmul_at", "gemm_matmul_at_swiglu_a", "gemm_matmul_t_ex", "gemm_matmul_at_ex",
    "gemm_matmul_at_swiglu_a_ex", "gemm_bwd_num_configs", "gemm_bwd_config_name", "gemm_bwd_select_config",
    "gemm_bwd_workspace_bytes", "gemm_matmul_t_swiglu_bwd", "gemm_matmul_t_swiglu_bwd_ex",
    "loss_cross_entropy", "loss_sum_losses", "loss_distill_cross_entropy", "act_ffn_swiglu_backward",
    "act_ffn_gelu_backward", "act_gelu_inplace", "attn_forward", "attn_backward",
    "attn_backward_workspace_bytes", "attn_qk_norm_rope",
    "attn_qk_norm_rope_backward", "attn_qk_norm_rope_workspace_bytes",
    "attn_qk_norm_rope_axes", "attn_qk_norm_rope_axes_backward",
    "attn_scored_forward", "attn_scored_backward", "attn_scored_backward_workspace_bytes",
    "block_norm", "block_norm_backward", "block_norm_backward_workspace_bytes",
    "gemm_timing_event_create", "gemm_timing_event_record", "gemm_timing_elapsed_ms", "gemm_timing_event_destroy",
)


class GemmOpts(ctypes.Structure):
    """struct gemm_opts of include/gemm_fwd.h."""
    _fields_ = [("config", ctypes.c_int64), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
                ("start_event", ctypes.c_void_p), ("stop_event", ctypes.c_void_p)]


def opts(config=-1, workspace=None, workspace_bytes=0, start=None, stop=None):
    """A gemm_opts passed by reference (ctypes.byref) to the _ex entry points."""
    return ctypes.byref(GemmOpts(-1 if config is None else int(config), workspace, int(workspace_bytes), start, stop))


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {status_string(status)} (status {status})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


SYNC_CHECK_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgemmfwd_sync.so")
_sync_lib = None


def load_library():
    """Load libgemmfwd.so (after torch, so both share torch's HIP runtime)."""
    global _lib
    if _lib is None:
        _lib = _open(_LIB_PATH)
    return _lib


def load_sync_check_library():
    """The verification build (same C ABI; see the race-check tests)."""
    global _sync_lib
    if _sync_lib is None:
        _sync_lib = _open(SYNC_CHECK_LIB_PATH)
    return _sync_lib


def _open(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    p, i64, u32, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int
    lib.gemm_fwd.argtypes = [p, p, p, p, i64, i64, i64, u32, p]
    lib.gemm_fwd.restype = c_int
    lib.gemm_fwd_swiglu.argtypes = [p, p, p, p, p, i64, i64, i64, c_int, p]
    lib.gemm_fwd_swiglu.restype = c_int
    o = ctypes.c_void_p  # const gemm_opts * (ctypes.byref or None)
    lib.gemm_fwd_ex.argtypes = [p, p, p, p, i64, i64, i64, u32, o, p]
    lib.gemm_fwd_ex.restype = c_int
    lib.gemm_fwd_swiglu_ex.argtypes = [p, p, p, p, p, i64, i64, i64, c_int, o, p]
    lib.gemm_fwd_swiglu_ex.restype = c_int
    lib.gemm_fwd_swiglu_noalloc.argtypes = [p, p, p, p, p, i64, i64, i64, c_int, p]
    lib.gemm_fwd_swiglu_noalloc.restype = c_int
    lib.gemm_fwd_workspace_bytes.argtypes = [i64, i64, i64, c_int, u32, c_int]
    lib.gemm_fwd_workspace_bytes.restype = i64
    lib.gemm_num_configs.argtypes = []
    lib.gemm_num_configs.restype = c_int
    lib.gemm_config_name.argtypes = [c_int]
    lib.gemm_config_name.restype = ctypes.c_char_p
    lib.gemm_select_config.argtypes = [i64, i64, i64, c_int, c_int, c_int]
    lib.gemm_select_config.restype = c_int
    lib.gemm_status_string.argtypes = [c_int]
    lib.gemm_status_string.restype = ctypes.c_char_p
    for name, n_in in (("gemm_matmul_t", 2), ("gemm_matmul_at", 2), ("gemm_matmul_at_swiglu_a", 3)):
        getattr(lib, name).argtypes = [p] * (n_in + 1) + [i64, i64, i64, u32, p]
        getattr(lib, name).restype = c_int
        getattr(lib, name + "_ex").argtypes = [p] * (n_in + 1) + [i64, i64, i64, u32, o, p]
        getattr(lib, name + "_ex").restype = c_int
    lib.gemm_matmul_t_swiglu_bwd.argtypes = [p] * 6 + [i64, i64, i64, p]
    lib.gemm_matmul_t_swiglu_bwd.restype = c_int
    lib.gemm_matmul_t_swiglu_bwd_ex.argtypes = [p] * 6 + [i64, i64, i64, o, p]
    lib.gemm_matmul_t_swiglu_bwd_ex.restype = c_int
    lib.gemm_bwd_workspace_bytes.argtypes = [c_int, i64, i64, i64, c_int, c_int]
    lib.gemm_bwd_workspace_bytes.restype = i64
    lib.gemm_bwd_num_configs.argtypes = []
    lib.gemm_bwd_num_configs.restype = c_int
    lib.gemm_bwd_config_name.argtypes = [c_int]
    lib.gemm_bwd_config_name.restype = ctypes.c_char_p
    lib.gemm_bwd_select_config.argtypes = [c_int, i64, i64, i64, c_int, c_int]
    lib.gemm_bwd_select_config.restype = c_int
    f32 = ctypes.c_float
    lib.loss_cross_entropy.argtypes = [p, p, p, i64, i64, f32, f32, f32, p]
    lib.loss_cross_entropy.restype = c_int
    lib.loss_sum_losses.argtypes = [p, p, i64, p]
    lib.loss_sum_losses.restype = c_int
    lib.act_ffn_swiglu_backward.argtypes = [p, p, p, p, p, i64, p]
    lib.act_ffn_swiglu_backward.restype = c_int
    lib.act_ffn_gelu_backward.argtypes = [p, p, p, i64, p]
    lib.act_ffn_gelu_backward.restype = c_int
    lib.act_gelu_inplace.argtypes = [p, p, i64, p]
    lib.act_gelu_inplace.restype = c_int
    for name in ("attn_forward", "attn_backward", "attn_qk_norm_rope", "attn_qk_norm_rope_backward",
                 "attn_qk_norm_rope_axes", "attn_qk_norm_rope_axes_backward", "loss_distill_cross_entropy",
                 "attn_scored_forward", "attn_scored_backward", "block_norm", "block_norm_backward"):
        getattr(lib, name).argtypes = [ctypes.c_char_p, p]  # the packed argument struct, the stream
        getattr(lib, name).restype = c_int
    lib.attn_backward_workspace_bytes.argtypes = [ctypes.c_char_p]
    lib.attn_backward_workspace_bytes.restype = i64
    lib.attn_qk_norm_rope_workspace_bytes.argtypes = [i64, i64]
    lib.attn_qk_norm_rope_workspace_bytes.restype = i64
    lib.attn_scored_backward_workspace_bytes.argtypes = [ctypes.c_char_p, c_int]
    lib.attn_scored_backward_workspace_bytes.restype = i64
    lib.block_norm_backward_workspace_bytes.argtypes = [ctypes.c_char_p]
    lib.block_norm_backward_workspace_bytes.restype = i64
    lib.gemm_timing_event_create.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
    lib.gemm_timing_event_create.restype = c_int
    lib.gemm_timing_event_record.argtypes = [p, p]
    lib.gemm_timing_event_record.restype = c_int
    lib.gemm_timing_elapsed_ms.argtypes = [p, p, ctypes.POINTER(f32)]
    lib.gemm_timing_elapsed_ms.restype = c_int
    lib.gemm_timing_event_destroy.argtypes = [p]
    lib.gemm_timing_event_destroy.restype = c_int
    return lib


class TimingEvent:
    """A timing event of the library (gemm_timing_event_create: no
    system-scope cache writeback when it is recorded) for the start_event /
    stop_event of gemm_opts; `handle` is what opts() takes."""

    def __init__(self):
        h = ctypes.c_void_p()
        st = load_library().gemm_timing_event_create(ctypes.byref(h))
        if st != 0:
            raise GemmError(st, "gemm_timing_event_create")
        self.handle = h.value

    def record(self, stream=None) -> None:
        """Record the event on `stream` (a torch stream or a raw handle;
        None: torch's current stream) as a marker between launches."""
        if stream is None:
            stream = torch.cuda.current_stream()
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        st = load_library().gemm_timing_event_record(self.handle, handle)
        if st != 0:
            raise GemmError(st, "gemm_timing_event_record")

    def elapsed_ms(self, stop: "TimingEvent") -> float:
        """Milliseconds from this event to `stop` (both recorded and complete)."""
        ms = ctypes.c_float()
        st = load_library().gemm_timing_elapsed_ms(self.handle, stop.handle, ctypes.byref(ms))
        if st != 0:
            raise GemmError(st, "gemm_timing_elapsed_ms")
        return ms.value

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.gemm_timing_event_destroy(self.handle)
            self.handle = None


def status_string(status: int) -> str:
    return load_library().gemm_status_string(int(status)).decode()


def num_configs() -> int:
    return load_library().gemm_num_configs()


def config_name(config: int):
    name = load_library().gemm_config_name(int(config))
    return None if name is None else name.decode()


def config_takes_w16(config: int) -> bool:
    """Whether forward configuration `config` has binary16-W kernels: the
    tiles that load W straight into the compute waves' registers (names
    ending in _wrN) are fp32-only, and the library refuses them binary16 W."""
    return "_wr" not in config_name(config)


def bwd_num_configs() -> int:
    return load_library().gemm_bwd_num_configs()


def bwd_config_name(config: int):
    name = load_library().gemm_bwd_config_name(int(config))
    return None if name is None else name.decode()


def bwd_kernel_config(op, M, K, N, swiglu=False, workspace=True) -> str:
    """Name of the configuration the library picks for a backward product
    (op "matmul_t" or "matmul_at"; M, K, N the forward's names), with or
    without a workspace."""
    code = {"matmul_t": 1, "matmul_at": 2}[op]
    return bwd_config_name(load_library().gemm_bwd_select_config(code, M, K, N, int(swiglu), int(workspace)))


def kernel_config(M, K, N, swiglu=False, w16=False, workspace=True) -> str:
    """Name of the tile configuration the library picks for a shape, with or
    without a workspace."""
    return config_name(load_library().gemm_select_config(M, K, N, int(swiglu), int(w16), int(workspace)))


# --- split-K workspaces ---
#
# The library holds no device memory: split-K partial tiles go to a
# workspace the caller provides.  The tensor-level calls below keep one
# zero-filled torch buffer per (device, stream), grown on demand; the library
# leaves a workspace zeroed after every call, and calls on one stream are
# ordered, so the buffer is reused as it is.  Calls on different streams get
# different buffers.

_workspaces = {}


def workspace(device, stream, nbytes):
    """(pointer, size) of the zero-filled workspace for `stream` on `device`,
    at least nbytes long; (None, 0) when nbytes is 0."""
    if nbytes <= 0:
        return None, 0
    key = (device.index, int(stream.cuda_stream))
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        with torch.cuda.stream(stream):
            # rounded up to a MiB: a few sizes serve every shape
            buf = torch.zeros(((nbytes + (1 << 20) - 1) >> 20) << 20, dtype=torch.uint8, device=device)
        _workspaces[key] = buf
    return buf.data_ptr(), buf.numel()


def _fwd_workspace(M, K, N, swiglu, w16, device, config):
    nbytes = load_library().gemm_fwd_workspace_bytes(M, K, N, int(swiglu), GEMM_FLAG_W_F16 if w16 else 0,
                                                     -1 if config is None else int(config))
    if nbytes < 0:
        raise GemmError(-2, "gemm_fwd_workspace_bytes")
    return workspace(device, torch.cuda.current_stream(device), nbytes)


# --- raw pointer-level calls (same names and argument order as the C ABI) ---

def gemm_fwd(X, W, R, Y, M, K, N, flags, stream) -> int:
    return load_library().gemm_fwd(X, W, R, Y, M, K, N, flags, stream)


def gemm_fwd_swiglu(G, U, W, R, Y, M, K, N, w_dtype, stream) -> int:
    return load_library().gemm_fwd_swiglu(G, U, W, R, Y, M, K, N, w_dtype, stream)


def gemm_fwd_ex(X, W, R, Y, M, K, N, flags, options, stream) -> int:
    return load_library().gemm_fwd_ex(X, W, R, Y, M, K, N, flags, options, stream)


def gemm_fwd_swiglu_ex(G, U, W, R, Y, M, K, N, w_dtype, options, stream) -> int:
    return load_library().gemm_fwd_swiglu_ex(G, U, W, R, Y, M, K, N, w_dtype, options, stream)


# --- tensor-level API ---

def _check_act(t, name, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda" or t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_w(W, K, device):
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise TypeError("W must be a 2-D torch.Tensor [K, N]")
    if W.device != device:
        raise ValueError(f"W must live on {device}, got {W.device}")
    if W.dtype not in (torch.float32, torch.float16):
        raise TypeError(f"W must be float32 or float16, got {W.dtype}")
    if not W.is_contiguous():
        raise ValueError("W must be contiguous (row-major [K, N])")
    if W.shape[0] != K:
        raise ValueError(f"W has {W.shape[0]} rows, expected K={K}")
    return W.shape[1]


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def matmul(X, W, R=None, out=None, config=None, use_workspace=True):
    """Y = X @ W (+ R).  X [M, K] f32, W [K, N] f32 or f16, R [M, N] f32 or None.
    config: a configuration index (None: the library's choice).  use_workspace:
    give the library the stream's split-K workspace (False: the plain
    gemm_fwd behaviour, no split-K)."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise TypeError("X must be a 2-D torch.Tensor [M, K]")
    M, K = X.shape
    device = X.device
    _check_act(X, "X", (M, K), device)
    N = _check_w(W, K, device)
    if R is not None:
        _check_act(R, "R", (M, N), device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=device)
    else:
        _check_act(out, "out", (M, N), device)
    w16 = W.dtype == torch.float16
    flags = GEMM_FLAG_W_F16 if w16 else 0
    ws, wsb = _fwd_workspace(M, K, N, False, w16, device, config) if use_workspace else (None, 0)
    st = gemm_fwd_ex(X.data_ptr(), W.data_ptr(), None if R is None else R.data_ptr(), out.data_ptr(),
                     M, K, N, flags, opts(config, ws, wsb), _stream(device))
    if st != 0:
        raise GemmError(st, "gemm_fwd_ex")
    return out


def matmul_residual(X, W, R, out=None, config=None, use_workspace=True):
    """Y = X @ W + R."""
    if R is None:
        raise ValueError("matmul_residual needs R")
    return matmul(X, W, R, out=out, config=config, use_workspace=use_workspace)


def matmul_residual_swiglu_a(G, U, W, R, out=None, config=None, use_workspace=True):
    """Y = (silu(G) * U) @ W + R, the SwiGLU combine fused into the A load
    (config and use_workspace as for matmul)."""
    if not isinstance(G, torch.Tensor) or G.dim() != 2:
        raise TypeError("G must be a 2-D torch.Tensor [M, K]")
    M, K = G.shape
    device = G.device
    _check_act(G, "G", (M, K), device)
    _check_act(U, "U", (M, K), device)
    N = _check_w(W, K, device)
    _check_act(R, "R", (M, N), device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=device)
    else:
        _check_act(out, "out", (M, N), device)
    w16 = W.dtype == torch.float16
    w_dtype = GEMM_W_F16 if w16 else GEMM_W_F32
    ws, wsb = _fwd_workspace(M, K, N, True, w16, device, config) if use_workspace else (None, 0)
    st = gemm_fwd_swiglu_ex(G.data_ptr(), U.data_ptr(), W.data_ptr(), R.data_ptr(), out.data_ptr(),
                            M, K, N, w_dtype, opts(config, ws, wsb), _stream(device))
    if st != 0:
        raise GemmError(st, "gemm_fwd_swiglu_ex")
    return out


# --- backward linear family (matmul_t, matmul_at and their _acc / _swiglu_a forms) ---

def _bwd_workspace(op, M, K, N, swiglu, device, config):
    nbytes = load_library().gemm_bwd_workspace_bytes(op, M, K, N, int(swiglu), -1 if config is None else int(config))
    if nbytes < 0:
        raise GemmError(-2, "gemm_bwd_workspace_bytes")
    return workspace(device, torch.cuda.current_stream(device), nbytes)


def _bwd_call(name, ptrs, M, K, N, acc, device, config, use_workspace=True):
    lib = load_library()
    flags = GEMM_FLAG_ACC if acc else 0
    op = 1 if name == "gemm_matmul_t" else 2
    ws, wsb = (_bwd_workspace(op, M, K, N, name.endswith("swiglu_a"), device, config) if use_workspace
               else (None, 0))
    st = getattr(lib, name + "_ex")(*ptrs, M, K, N, flags, opts(config, ws, wsb), _stream(device))
    if st != 0:
        raise GemmError(st, name)


def _out(out, shape, device, acc):
    if out is None:
        if acc:
            raise ValueError("accumulation needs the output tensor")
        return torch.empty(shape, dtype=torch.float32, device=device)
    _check_act(out, "out", shape, device)
    return out


def matmul_t(dY, W, out=None, acc=False, config=None, use_workspace=True):
    """dX = dY @ W^T (matmul_t), or out += dY @ W^T with acc=True (matmul_t_acc).
    dY [M, N] f32, W [K, N] f32 (the forward's weight); dX [M, K]."""
    if not isinstance(dY, torch.Tensor) or dY.dim() != 2:
        raise TypeError("dY must be a 2-D torch.Tensor [M, N]")
    M, N = dY.shape
    device = dY.device
    _check_act(dY, "dY", (M, N), device)
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise TypeError("W must be a 2-D torch.Tensor [K, N]")
    K = W.shape[0]
    _check_act(W, "W", (K, N), device)
    out = _out(out, (M, K), device, acc)
    _bwd_call("gemm_matmul_t", (dY.data_ptr(), W.data_ptr(), out.data_ptr()), M, K, N, acc, device, config,
              use_workspace)
    return out


def matmul_at(X, dY, out=None, acc=False, config=None, use_workspace=True):
    """dW = X^T @ dY (matmul_at), or out += X^T @ dY with acc=True (matmul_at_acc).
    X [M, K] f32, dY [M, N] f32; dW [K, N]."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise TypeError("X must be a 2-D torch.Tensor [M, K]")
    M, K = X.shape
    device = X.device
    _check_act(X, "X", (M, K), device)
    if not isinstance(dY, torch.Tensor) or dY.dim() != 2:
        raise TypeError("dY must be a 2-D torch.Tensor [M, N]")
    N = dY.shape[1]
    _check_act(dY, "dY", (M, N), device)
    out = _out(out, (K, N), device, acc)
    _bwd_call("gemm_matmul_at", (X.data_ptr(), dY.data_ptr(), out.data_ptr()), M, K, N, acc, device, config,
              use_workspace)
    return out


def matmul_at_swiglu_a(G, U, dY, out=None, acc=False, config=None, use_workspace=True):
    """dW = (silu(G) * U)^T @ dY (matmul_at_swiglu_a), or out += ... with acc=True
    (matmul_at_acc_swiglu_a); the combine is recomputed as A is staged.
    G, U [M, K] f32, dY [M, N] f32; dW [K, N]."""
    if not isinstance(G, torch.Tensor) or G.dim() != 2:
        raise TypeError("G must be a 2-D torch.Tensor [M, K]")
    M, K = G.shape
    device = G.device
    _check_act(G, "G", (M, K), device)
    _check_act(U, "U", (M, K), device)
    if not isinstance(dY, torch.Tensor) or dY.dim() != 2:
        raise TypeError("dY must be a 2-D torch.Tensor [M, N]")
    N = dY.shape[1]
    _check_act(dY, "dY", (M, N), device)
    out = _out(out, (K, N), device, acc)
    _bwd_call("gemm_matmul_at_swiglu_a", (G.data_ptr(), U.data_ptr(), dY.data_ptr(), out.data_ptr()),
              M, K, N, acc, device, config, use_workspace)
    return out


def matmul_t_swiglu_backward(dY, W, G, U, grad_gate=None, grad_up=None, config=None):
    """The FFN down-projection's input gradient dH = dY @ W^T turned straight
    into the SwiGLU gradients (dH itself is never stored):
    grad_gate = nan_guard(dH * U * silu'(G)), grad_up = nan_guard(dH * silu(G)).
    dY [M, N], W [K, N] (the forward weight), G, U [M, K] f32.
    Returns (grad_gate, grad_up); either may be given as G or U to overwrite it."""
    if not isinstance(dY, torch.Tensor) or dY.dim() != 2:
        raise TypeError("dY must be a 2-D torch.Tensor [M, N]")
    M, N = dY.shape
    device = dY.device
    _check_act(dY, "dY", (M, N), device)
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise TypeError("W must be a 2-D torch.Tensor [K, N]")
    K = W.shape[0]
    _check_act(W, "W", (K, N), device)
    _check_act(G, "G", (M, K), device)
    _check_act(U, "U", (M, K), device)
    grad_gate = torch.empty((M, K), dtype=torch.float32, device=device) if grad_gate is None else grad_gate
    grad_up = torch.empty((M, K), dtype=torch.float32, device=device) if grad_up is None else grad_up
    _check_act(grad_gate, "grad_gate", (M, K), device)
    _check_act(grad_up, "grad_up", (M, K), device)
    lib = load_library()
    ptrs = (dY.data_ptr(), W.data_ptr(), G.data_ptr(), U.data_ptr(), grad_gate.data_ptr(), grad_up.data_ptr())
    ws, wsb = _bwd_workspace(1, M, K, N, False, device, config)
    st = lib.gemm_matmul_t_swiglu_bwd_ex(*ptrs, M, K, N, opts(config, ws, wsb), _stream(device))
    if st != 0:
        raise GemmError(st, "gemm_matmul_t_swiglu_bwd_ex")
    return grad_gate, grad_up


# --- fused loss (include/loss.h) ---

def cross_entropy(logits, targets, alpha=0.0, beta=0.0, inv_norm=None, losses=None):
    """cross_entropy: per-row losses, and the gradient written over `logits`
    in place.  logits [S, V] f32, targets [S] int32/int64 (values >= V, or
    negative, mark ignored rows); inv_norm defaults to 1 / (number of rows
    with a target in [0, V)), which reads that count back to the host.
    Returns the losses [S] f32 tensor."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise TypeError("logits must be a 2-D torch.Tensor [S, V]")
    S, V = logits.shape
    device = logits.device
    _check_act(logits, "logits", (S, V), device)
    if not isinstance(targets, torch.Tensor) or tuple(targets.shape) != (S,) or targets.device != device:
        raise ValueError(f"targets must be a [{S}] tensor on {device}")
    if targets.dtype not in (torch.int32, torch.int64):
        raise TypeError("targets must be int32 or int64")
    # the kernel reads targets as uint32: a negative value reads as >= V and
    # marks an ignored row, like any other out-of-range target
    t32 = targets if targets.dtype == torch.int32 and targets.is_contiguous() else targets.to(torch.int32).contiguous()
    if inv_norm is None:
        valid = int(((targets >= 0) & (targets < V)).sum().item())
        inv_norm = 1.0 / valid if valid else 0.0
    if losses is None:
        losses = torch.empty((S,), dtype=torch.float32, device=device)
    else:
        _check_act(losses, "losses", (S,), device)
    st = load_library().loss_cross_entropy(logits.data_ptr(), t32.data_ptr(), losses.data_ptr(), S, V,
                                           float(alpha), float(beta), float(inv_norm), _stream(device))
    if st != 0:
        raise GemmError(st, "loss_cross_entropy")
    return losses


def sum_losses(losses, out=None):
    """sum_losses: the scalar total of the per-row losses, as a [1] tensor."""
    if not isinstance(losses, torch.Tensor) or losses.dim() != 1:
        raise TypeError("losses must be a 1-D torch.Tensor")
    device = losses.device
    _check_act(losses, "losses", tuple(losses.shape), device)
    if out is None:
        out = torch.empty((1,), dtype=torch.float32, device=device)
    else:
        _check_act(out, "out", (1,), device)
    st = load_library().loss_sum_losses(losses.data_ptr(), out.data_ptr(), losses.shape[0], _stream(device))
    if st != 0:
        raise GemmError(st, "loss_sum_losses")
    return out


# --- distillation (include/distill.h) ---

_DISTILL_ARGS = struct.Struct("=6q 3q 3q 5d")


def _call_packed(name, args, device):
    """Enqueue `name` on `device`'s current stream, with that device current.
    `args` is the entry point's argument struct, packed field by field (every
    field is 8 bytes wide: pointers, int64_t, double)."""
    fn = getattr(load_library(), name)
    # the handle alone: a torch stream object around it costs 1.8 us a call
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch._C._cuda_getDevice():
        st = fn(args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(args, stream)
    if st != 0:
        raise GemmError(st, name)


def _indices(t, name, shape, device):
    """(pointer, 1 if int64) of a dense index tensor."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor on {device}")
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    return t.data_ptr(), 1 if t.dtype == torch.int64 else 0


def distill_cross_entropy(logits, targets, teacher_ids, teacher_logits, temperature=1.0, mix=0.5, alpha=0.0, beta=0.0,
                          inv_norm=None, dlogits=None, losses=None):
    """cross_entropy mixed with distillation from a teacher's best logits: the
    losses of every row, and the gradient of inv_norm * sum over rows of
    (1 - mix) * cross-entropy + mix * distillation.

    logits [S, V] f32; targets [S] int32/int64 (a value outside [0, V) marks a
    padding row; None only with mix 1); teacher_ids [S, K] int32/int64 and
    teacher_logits [S, K] f32/f16, K up to 1024, the teacher's columns and its
    logits there (an id outside [0, V) marks an unused entry).  The
    distillation loss is temperature^2 * KL(teacher over its entries ||
    student over the vocabulary), both at the temperature; alpha and beta are
    cross_entropy's label smoothing and z-loss.  inv_norm defaults to 1 /
    (number of rows that are not padding), which reads that count back to the
    host when there are targets.  The gradient is written to dlogits, or over
    `logits` when that is None.  Returns the losses [2, S]: cross-entropy and
    distillation."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise TypeError("logits must be a 2-D torch.Tensor [S, V]")
    S, V = logits.shape
    device = logits.device
    _check_act(logits, "logits", (S, V), device)
    if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2:
        raise TypeError("teacher_ids must be a 2-D torch.Tensor [S, K]")
    K = teacher_ids.shape[1]
    pi, ids64 = _indices(teacher_ids, "teacher_ids", (S, K), device)
    if not isinstance(teacher_logits, torch.Tensor) or teacher_logits.shape != (S, K) \
            or teacher_logits.device != device or not teacher_logits.is_contiguous():
        raise ValueError(f"teacher_logits must be a contiguous [{S}, {K}] tensor on {device}")
    if teacher_logits.dtype not in (torch.float32, torch.float16):
        raise TypeError(f"teacher_logits must be float32 or float16, got {teacher_logits.dtype}")
    pt, targets64 = (0, 0) if targets is None else _indices(targets, "targets", (S,), device)
    if targets is None and mix != 1:
        raise ValueError("targets may be None only with mix 1")
    if inv_norm is None:
        valid = S if targets is None else int(((targets >= 0) & (targets < V)).sum().item())
        inv_norm = 1.0 / valid if valid else 0.0
    if dlogits is None:
        dlogits = logits
    else:
        _check_act(dlogits, "dlogits", (S, V), device)
    if losses is None:
        losses = torch.empty((2, S), dtype=torch.float32, device=device)
    else:
        _check_act(losses, "losses", (2, S), device)
    _call_packed("loss_distill_cross_entropy",
                 _DISTILL_ARGS.pack(logits.data_ptr(), dlogits.data_ptr(), pt, pi, teacher_logits.data_ptr(),
                                    losses.data_ptr(), targets64, ids64,
                                    1 if teacher_logits.dtype == torch.float16 else 0, S, V, K, float(temperature),
                                    float(mix), float(alpha), float(beta), float(inv_norm)), device)
    return losses


# --- FFN activation kernels (include/activation.h) ---

def _same_shape(name, t, ref):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 torch.Tensor")
    if t.device != ref.device or t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {tuple(ref.shape)} on {ref.device}")


def ffn_swiglu_backward(grad_hidden, gate, up, grad_gate=None, grad_up=None):
    """grad_gate = nan_guard(g * up * silu'(gate)), grad_up = nan_guard(g * silu(gate)),
    element-wise over tensors of one shape.  Returns (grad_gate, grad_up)."""
    _same_shape("grad_hidden", grad_hidden, grad_hidden)
    _same_shape("gate", gate, grad_hidden)
    _same_shape("up", up, grad_hidden)
    grad_gate = torch.empty_like(gate) if grad_gate is None else grad_gate
    grad_up = torch.empty_like(up) if grad_up is None else grad_up
    _same_shape("grad_gate", grad_gate, grad_hidden)
    _same_shape("grad_up", grad_up, grad_hidden)
    st = load_library().act_ffn_swiglu_backward(grad_hidden.data_ptr(), gate.data_ptr(), up.data_ptr(),
                                                grad_gate.data_ptr(), grad_up.data_ptr(), grad_hidden.numel(),
                                                _stream(grad_hidden.device))
    if st != 0:
        raise GemmError(st, "act_ffn_swiglu_backward")
    return grad_gate, grad_up


def ffn_gelu_backward(grad_hidden, pre_gelu, grad_pre=None):
    """grad_pre = nan_guard(g * gelu'(pre_gelu)), element-wise."""
    _same_shape("grad_hidden", grad_hidden, grad_hidden)
    _same_shape("pre_gelu", pre_gelu, grad_hidden)
    grad_pre = torch.empty_like(pre_gelu) if grad_pre is None else grad_pre
    _same_shape("grad_pre", grad_pre, grad_hidden)
    st = load_library().act_ffn_gelu_backward(grad_hidden.data_ptr(), pre_gelu.data_ptr(), grad_pre.data_ptr(),
                                              grad_hidden.numel(), _stream(grad_hidden.device))
    if st != 0:
        raise GemmError(st, "act_ffn_gelu_backward")
    return grad_pre


def gelu_inplace(x, pre_gelu=None):
    """x = gelu(x) in place (tanh approximation); pre_gelu, if given, receives
    the input values.  Returns x."""
    _same_shape("x", x, x)
    if pre_gelu is not None:
        _same_shape("pre_gelu", pre_gelu, x)
    st = load_library().act_gelu_inplace(x.data_ptr(), None if pre_gelu is None else pre_gelu.data_ptr(), x.numel(),
                                         _stream(x.device))
    if st != 0:
        raise GemmError(st, "act_gelu_inplace")
    return x


# --- attention (include/attention.h) ---

_FORWARD_ARGS = struct.Struct("=8qd 12q q")
_PROBLEM = struct.Struct("=8qd")
_BACKWARD_ARGS = struct.Struct("=8qd 15q q 9q 2q")
_SCORED_ARGS = struct.Struct("=8qd d2q 12q q")
_SCORED_BACKWARD_ARGS = struct.Struct("=8qd d2q 15q q 9q q 2q")
_NORM_ARGS = struct.Struct("=11qd 12q")
_NORM_BACKWARD_ARGS = struct.Struct("=11qd 18q 4q")
_NORM_AXES_ARGS = struct.Struct("=11qd 2q 12q")
_NORM_AXES_BACKWARD_ARGS = struct.Struct("=11qd 2q 18q 4q")


def _heads(t, name, shape, device):
    """(pointer, token stride, head stride) of the [tokens, heads, head_dim] tensor t."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must live on {device if device.type == 'cuda' else 'a GPU'}, got {t.device}")
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st, sh, sd = t.stride()
    if sd != 1 and shape[2] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), st, sh


def _out_heads(t, name, shape, like):
    """A result and its fields as of _heads: t itself, checked, or where that
    is None a new dense one on `like`'s device, which needs no check."""
    if t is not None:
        return t, _heads(t, name, shape, like.device)
    t = like.new_empty(shape)
    return t, (t.data_ptr(), shape[1] * shape[2], shape[2])


def _out_vector(t, name, like):
    """The same for a vector as long as the checked vector `like`, and its pointer."""
    if t is not None:
        return t, _vector(t, name, like.device, like.shape[0])
    t = torch.empty_like(like)
    return t, t.data_ptr()


def _row_values(t, name, shape, device):
    """Pointer of a dense float32 [heads, tokens] tensor."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.float32 or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _cu_seqlens(cu_seqlens, device):
    """(pointer, sequences) of the sequences' bounds; (0, 0) for None."""
    if cu_seqlens is None:
        return 0, 0
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.device != device \
            or cu_seqlens.shape[0] < 1 or not cu_seqlens.is_contiguous():
        raise ValueError(f"cu_seqlens must be a contiguous 1-D tensor of at least one entry on {device}")
    if cu_seqlens.dtype != torch.int32:
        raise TypeError(f"cu_seqlens must be int32, got {cu_seqlens.dtype}")
    return cu_seqlens.data_ptr(), cu_seqlens.shape[0] - 1


def _attn_problem(q, k, cu_seqlens, causal, window, scale):
    """The fields of attn_problem, and the shapes of q and of k and v."""
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise TypeError(f"{name} must be a 3-D torch.Tensor [tokens, heads, head_dim]")
    tokens, hq, dim = shape_q = q.shape
    hkv = k.shape[1]
    if hq < 1 or hkv < 1 or hq % hkv:
        raise ValueError(f"{hq} query heads do not share {hkv} key/value heads evenly")
    cu, nseq = _cu_seqlens(cu_seqlens, q.device)
    if window < 0:
        raise ValueError(f"window must not be negative, got {window}")
    if scale is None:
        scale = dim ** -0.5 if dim else 1.0
    return (cu, nseq, tokens, hq, hkv, dim, 1 if causal else 0, int(window), float(scale)), shape_q, (tokens, hkv, dim)


def _attn_scores(problem, softcap, slopes, prefix_lens, device):
    """The fields of attn_scores, or None for plain scores."""
    if softcap == 0 and slopes is None and prefix_lens is None:
        return None
    _, nseq, _, hq, _, _, causal, _, _ = problem
    pp = 0
    if prefix_lens is not None:
        n = nseq if problem[0] else 1
        if not isinstance(prefix_lens, torch.Tensor) or prefix_lens.shape != (n,) or prefix_lens.device != device \
                or not prefix_lens.is_contiguous():
            raise ValueError(f"prefix_lens must be a contiguous [{n}] tensor on {device}")
        if prefix_lens.dtype != torch.int32:
            raise TypeError(f"prefix_lens must be int32, got {prefix_lens.dtype}")
        if not causal:
            raise ValueError("prefix_lens needs causal: without it all keys are seen anyway")
        pp = prefix_lens.data_ptr()
    return float(softcap), 0 if slopes is None else _vector(slopes, "slopes", device, hq), pp


def attention(q, k, v, cu_seqlens=None, causal=True, window=0, scale=None, out=None, lse=None, softcap=0.0, slopes=None,
              prefix_lens=None):
    """Attention over packed sequences: out = softmax(scale q k^T over the
    visible keys) v, and lse, the logarithm of each row's sum of exponentials,
    which attention_backward needs.

    q [tokens, q_heads, head_dim], k and v [tokens, kv_heads, head_dim]
    float32 (q_heads a multiple of kv_heads, head_dim a multiple of 4 up to
    128), contiguous along the head with any strides that are multiples of 4,
    so the projection's output is taken as views.  cu_seqlens, int32
    [sequences + 1] on the device: sequence b is rows cu_seqlens[b] to
    cu_seqlens[b + 1] - 1 (None: all rows are one sequence); rows of no
    sequence get out 0 and lse -inf.  A row sees the rows of its sequence, up
    to itself with causal, less than `window` away with window > 0.  scale
    defaults to head_dim ** -0.5.  out may be q itself.

    Scores of other forms, in any combination: softcap > 0 (1e-6 to 1e6)
    bends them to softcap * tanh(score / softcap); slopes, float32 [q_heads],
    takes slopes[head] * |i - j| from them; prefix_lens, int32 [sequences] on
    the device ([1] without cu_seqlens), lets every row of sequence b see its
    first prefix_lens[b] rows too (with causal).
    Returns (out like q, lse [q_heads, tokens])."""
    problem, shape_q, shape_k = _attn_problem(q, k, cu_seqlens, causal, window, scale)
    device = q.device
    tq = _heads(q, "q", shape_q, device)
    tk = _heads(k, "k", shape_k, device)
    tv = _heads(v, "v", shape_k, device)
    tokens, hq, _ = shape_q
    out, to = _out_heads(out, "out", shape_q, q)
    if lse is None:
        lse = q.new_empty((hq, tokens))
        pl = lse.data_ptr()
    else:
        pl = _row_values(lse, "lse", (hq, tokens), device)
    scores = _attn_scores(problem, softcap, slopes, prefix_lens, device)
    if scores is None:
        _call_packed("attn_forward", _FORWARD_ARGS.pack(*problem, *tq, *tk, *tv, *to, pl), device)
    else:
        _call_packed("attn_scored_forward", _SCORED_ARGS.pack(*problem, *scores, *tq, *tk, *tv, *to, pl), device)
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_seqlens=None, causal=True, window=0, scale=None, dq=None, dk=None,
                       dv=None, softcap=0.0, slopes=None, prefix_lens=None, dslopes=None):
    """Gradients of attention: dq, dk, dv from dout, its inputs, and the out
    and lse it returned (the probabilities are formed again from lse).
    Arguments as for attention; dq, dk and dv may be views of one buffer, but
    may not overlap an input.  Rows of no sequence get zero gradients.
    dslopes, float32 [q_heads], gets the gradient of slopes where it is given.
    Returns (dq, dk, dv), and dslopes behind them where it is given."""
    problem, shape_q, shape_k = _attn_problem(q, k, cu_seqlens, causal, window, scale)
    device = q.device
    tg = _heads(dout, "dout", shape_q, device)
    tq = _heads(q, "q", shape_q, device)
    tk = _heads(k, "k", shape_k, device)
    tv = _heads(v, "v", shape_k, device)
    to = _heads(out, "out", shape_q, device)
    pl = _row_values(lse, "lse", (shape_q[1], shape_q[0]), device)
    dq, tdq = _out_heads(dq, "dq", shape_q, q)
    dk, tdk = _out_heads(dk, "dk", shape_k, q)
    dv, tdv = _out_heads(dv, "dv", shape_k, q)
    scores = _attn_scores(problem, softcap, slopes, prefix_lens, device)
    if dslopes is not None and slopes is None:
        raise ValueError("dslopes needs slopes")
    # less than 0 for a problem that the call below refuses, with the reason
    if scores is None:
        nbytes = max(0, load_library().attn_backward_workspace_bytes(_PROBLEM.pack(*problem)))
    else:
        pd = 0 if dslopes is None else _vector(dslopes, "dslopes", device, shape_q[1])
        nbytes = max(0, load_library().attn_scored_backward_workspace_bytes(_PROBLEM.pack(*problem), 1 if pd else 0))
    # scratch of this call's own: two captured graphs share nothing
    scratch = q.new_empty((nbytes // 4,)) if nbytes else None
    ps = scratch.data_ptr() if nbytes else 0
    if scores is None:
        _call_packed("attn_backward",
                     _BACKWARD_ARGS.pack(*problem, *tg, *tq, *tk, *tv, *to, pl, *tdq, *tdk, *tdv, ps, nbytes), device)
        return dq, dk, dv
    _call_packed("attn_scored_backward",
                 _SCORED_BACKWARD_ARGS.pack(*problem, *scores, *tg, *tq, *tk, *tv, *to, pl, *tdq, *tdk, *tdv, pd, ps,
                                            nbytes), device)
    return (dq, dk, dv) if dslopes is None else (dq, dk, dv, dslopes)


def _vector(t, name, device, n=None):
    """Pointer of a dense float32 vector (of n values)."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.float32 or t.dim() != 1 \
            or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a contiguous float32 vector{'' if n is None else f' of {n}'} on {device}")
    return t.data_ptr()


def _attn_norm(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, pair_axis):
    """The fields of attn_norm and, with pair_axis, of attn_axes, and the shapes of q and of k."""
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise TypeError(f"{name} must be a 3-D torch.Tensor [tokens, heads, head_dim]")
    device = q.device
    tokens, hq, dim = q.shape
    hk = k.shape[1]
    by_axis = pair_axis is not None
    if not isinstance(positions, torch.Tensor) or positions.dim() != (2 if by_axis else 1) \
            or positions.shape[-1] != tokens or positions.device != device or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous [{'axes, ' if by_axis else ''}{tokens}] tensor on {device}")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    pf = _vector(inv_freq, "inv_freq", device)
    rotated = 2 * inv_freq.shape[0]
    if rotated > dim:
        raise ValueError(f"inv_freq has {rotated // 2} entries, a head only {dim} dimensions")
    fields = (positions.data_ptr(), 1 if positions.dtype == torch.int64 else 0, pf,
              _vector(q_weight, "q_weight", device, dim), _vector(k_weight, "k_weight", device, dim), tokens, hq, hk,
              dim, rotated, 1 if interleaved else 0, float(eps))
    if by_axis:
        if not isinstance(pair_axis, torch.Tensor) or pair_axis.shape != inv_freq.shape or pair_axis.device != device \
                or not pair_axis.is_contiguous():
            raise ValueError(f"pair_axis must be a contiguous [{rotated // 2}] tensor on {device}")
        if pair_axis.dtype != torch.int32:
            raise TypeError(f"pair_axis must be int32, got {pair_axis.dtype}")
        fields += (pair_axis.data_ptr(), positions.shape[0])
    return fields, q.shape, (tokens, hk, dim)


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, interleaved=False, q_out=None, k_out=None,
                 pair_axis=None):
    """Root-mean-square norm of every query and key head, times a weight, then
    the rotation by the token's position, in one pass over both.

    q [tokens, q_heads, head_dim] and k [tokens, k_heads, head_dim] float32,
    contiguous along the head with any other strides (head_dim even, up to
    256); q_weight, k_weight [head_dim]; positions int32 or int64 [tokens];
    inv_freq float32 [rotated / 2]: pair p of the first `rotated` dimensions
    turns by positions * inv_freq[p].  Pair p is dimensions p and p + rotated
    / 2, or with interleaved 2p and 2p + 1.  q_out and k_out may be q and k.
    With pair_axis, int32 [rotated / 2], positions is [axes, tokens] (the
    time, height and width of a patch, say) and pair p turns by
    positions[pair_axis[p]] * inv_freq[p]; sections of neighbouring pairs, or
    axes in turn, are a matter of that array (on the device, its entries in
    [0, axes)).
    Returns (q_out, k_out)."""
    fields, shape_q, shape_k = _attn_norm(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, pair_axis)
    device = q.device
    tq = _heads(q, "q", shape_q, device)
    tk = _heads(k, "k", shape_k, device)
    q_out, toq = _out_heads(q_out, "q_out", shape_q, q)
    k_out, tok = _out_heads(k_out, "k_out", shape_k, q)
    if pair_axis is None:
        _call_packed("attn_qk_norm_rope", _NORM_ARGS.pack(*fields, *tq, *tk, *toq, *tok), device)
    else:
        _call_packed("attn_qk_norm_rope_axes", _NORM_AXES_ARGS.pack(*fields, *tq, *tk, *toq, *tok), device)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, interleaved=False,
                          dq=None, dk=None, dq_weight=None, dk_weight=None, pair_axis=None):
    """Gradients of qk_norm_rope, from those of its results and its inputs.
    dq may be dq_out or q, dk may be dk_out or k (which are overwritten).
    Returns (dq, dk, dq_weight, dk_weight); the weights' gradients are sums
    over all tokens and heads."""
    fields, shape_q, shape_k = _attn_norm(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, pair_axis)
    device = q.device
    tgq = _heads(dq_out, "dq_out", shape_q, device)
    tgk = _heads(dk_out, "dk_out", shape_k, device)
    tq = _heads(q, "q", shape_q, device)
    tk = _heads(k, "k", shape_k, device)
    dq, tdq = _out_heads(dq, "dq", shape_q, q)
    dk, tdk = _out_heads(dk, "dk", shape_k, q)
    tokens, _, dim = shape_q
    dq_weight, pqw = _out_vector(dq_weight, "dq_weight", q_weight)
    dk_weight, pkw = _out_vector(dk_weight, "dk_weight", k_weight)
    nbytes = load_library().attn_qk_norm_rope_workspace_bytes(tokens, dim)
    if nbytes < 0:
        raise GemmError(-2, "attn_qk_norm_rope_workspace_bytes")
    # scratch of this call's own: two captured graphs share nothing
    scratch = q.new_empty((nbytes // 4,))
    name, args = (("attn_qk_norm_rope_backward", _NORM_BACKWARD_ARGS) if pair_axis is None else
                  ("attn_qk_norm_rope_axes_backward", _NORM_AXES_BACKWARD_ARGS))
    _call_packed(name, args.pack(*fields, *tgq, *tgk, *tq, *tk, *tdq, *tdk, pqw, pkw, scratch.data_ptr(), nbytes),
                 device)
    return dq, dk, dq_weight, dk_weight


# --- norms around a block (include/block_norm.h) ---

_BLOCK_ARGS = struct.Struct("=9q3d 8q")
_BLOCK_PROBLEM = struct.Struct("=9q3d")
_BLOCK_BACKWARD_ARGS = struct.Struct("=9q3d 12q 4q 2q")


def _rows(t, name, shape, device):
    """(pointer, row stride) of the [tokens, width] tensor t; (0, 0) for None."""
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must live on {device if device.type == 'cuda' else 'a GPU'}, got {t.device}")
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st, sd = t.stride()
    if sd != 1 and shape[1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), st


def _out_rows(t, name, shape, like):
    """As _out_heads for [tokens, width]."""
    if t is not None:
        return t, _rows(t, name, shape, like.device)
    # dense like `like` itself where that is dense, which takes torch 0.5 us less
    t = torch.empty_like(like) if like.is_contiguous() else like.new_empty(shape)
    return t, (t.data_ptr(), shape[1])


def _gate(t, name, shape, device):
    """(pointer, row stride) of a [width] or [sequences, width] tensor with contiguous rows."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.device != device or t.dtype != torch.float32 \
            or (t.stride(-1) != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be a float32 tensor of shape {tuple(shape)} on {device} with contiguous rows")
    return t.data_ptr(), t.stride(0)


def _block_problem(rows, name, pre_weight, post_weight, gate, residual_scale, block_scale, cu_seqlens, eps):
    """The fields of block_norm_problem for the [tokens, width] tensor `rows`, and the gate's shape."""
    if not isinstance(rows, torch.Tensor) or rows.dim() != 2:
        raise TypeError(f"{name} must be a 2-D torch.Tensor [tokens, width]")
    device = rows.device
    tokens, width = rows.shape
    cu, nseq = _cu_seqlens(cu_seqlens, device)
    by_seq, shape_gate, pg, gate_st = 0, None, 0, 0
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dim() not in (1, 2):
            raise TypeError("gate must be a torch.Tensor [width] or [sequences, width]")
        by_seq = gate.dim() - 1
        if by_seq and cu_seqlens is None:
            raise ValueError("a gate for each sequence needs cu_seqlens")
        shape_gate = torch.Size((nseq, width) if by_seq else (width,))
        pg, gate_st = _gate(gate, "gate", shape_gate, device)
    fields = (0 if pre_weight is None else _vector(pre_weight, "pre_weight", device, width),
              0 if post_weight is None else _vector(post_weight, "post_weight", device, width), pg, by_seq, gate_st, cu, nseq,
              tokens, width, float(residual_scale), float(block_scale), float(eps))
    return fields, shape_gate


def block_norm(x, y=None, pre_weight=None, post_weight=None, gate=None, residual_scale=1.0, block_scale=1.0,
               cu_seqlens=None, eps=1e-6, x_out=None, h_out=None):
    """The norm behind a block, its gate, the update of the residual stream
    and the norm in front of the next block, in one pass:

        n = norm(y) * post_weight                 (y without post_weight)
        x_out = residual_scale * x + block_scale * gate * n
        h = norm(x_out) * pre_weight              (None without pre_weight)

    where norm divides a row by its root mean square.  x, the residual stream,
    and y, the block's output, are [tokens, width] float32 with contiguous
    rows at any stride, width up to 8192.  gate is [width], or [sequences,
    width], rows at any stride, with cu_seqlens (int32 [sequences + 1] on the
    device, as for attention; rows of no sequence get x_out and h 0), or None
    for 1.  Without
    y (in front of the first block, behind the last) x_out is x and only the
    norm is formed.  x_out and h_out may each be x or y.
    Returns (x_out, h)."""
    fields, _ = _block_problem(x, "x", pre_weight, post_weight, gate, residual_scale, block_scale, cu_seqlens, eps)
    device, shape = x.device, x.shape
    if y is None and (pre_weight is None or x_out is not None or post_weight is not None or gate is not None
                      or residual_scale != 1 or block_scale != 1):
        raise ValueError("without y there is only the norm: pre_weight, and no x_out, post_weight, gate or scale")
    if pre_weight is None and h_out is not None:
        raise ValueError("h_out needs pre_weight")
    tx, ty = _rows(x, "x", shape, device), _rows(y, "y", shape, device)
    txo = th = (0, 0)
    if y is not None:
        x_out, txo = _out_rows(x_out, "x_out", shape, x)
    if pre_weight is not None:
        h_out, th = _out_rows(h_out, "h_out", shape, x)
    _call_packed("block_norm", _BLOCK_ARGS.pack(*fields, *tx, *ty, *txo, *th), device)
    return x if y is None else x_out, h_out


def block_norm_backward(dx_out, dh, x_out, y=None, pre_weight=None, post_weight=None, gate=None, residual_scale=1.0,
                        block_scale=1.0, cu_seqlens=None, eps=1e-6, dx=None, dy=None, dpre_weight=None,
                        dpost_weight=None, dgate=None):
    """Gradients of block_norm, from those of its results, dx_out (of the
    residual stream, from what reads it later; None counts as zero) and dh,
    and from x_out and y.  Other arguments as for block_norm; dx and dy may
    each be dx_out, dh, x_out or y.
    Returns (dx, dy, dpre_weight, dpost_weight, dgate), None for what the call
    has none of."""
    fields, shape_gate = _block_problem(x_out, "x_out", pre_weight, post_weight, gate, residual_scale, block_scale,
                                        cu_seqlens, eps)
    device, shape = x_out.device, x_out.shape
    if y is None and (pre_weight is None or dy is not None or post_weight is not None or gate is not None
                      or residual_scale != 1 or block_scale != 1):
        raise ValueError("without y there is only the norm: pre_weight, and no dy, post_weight, gate or scale")
    if (dh is None) != (pre_weight is None):
        raise ValueError("dh and pre_weight belong together")
    if dx_out is None and pre_weight is None:
        raise ValueError("without pre_weight there is dx_out")
    if (pre_weight is None and dpre_weight is not None) or (post_weight is None and dpost_weight is not None) \
            or (gate is None and dgate is not None):
        raise ValueError("dpre_weight, dpost_weight and dgate need pre_weight, post_weight and gate")
    inputs = (*_rows(dx_out, "dx_out", shape, device), *_rows(dh, "dh", shape, device),
              *_rows(x_out, "x_out", shape, device), *_rows(y, "y", shape, device))
    tdy, ppre, ppost, pgate, dgate_st = (0, 0), 0, 0, 0, 0
    dx, tdx = _out_rows(dx, "dx", shape, x_out)
    if y is not None:
        dy, tdy = _out_rows(dy, "dy", shape, x_out)
    if pre_weight is not None:
        dpre_weight, ppre = _out_vector(dpre_weight, "dpre_weight", pre_weight)
    if post_weight is not None:
        dpost_weight, ppost = _out_vector(dpost_weight, "dpost_weight", post_weight)
    if gate is not None:
        if dgate is None:
            dgate = gate.new_empty(shape_gate)
        pgate, dgate_st = _gate(dgate, "dgate", shape_gate, device)
    nbytes = load_library().block_norm_backward_workspace_bytes(_BLOCK_PROBLEM.pack(*fields))
    # scratch of this call's own: two captured graphs share nothing (none for
    # a problem that the call below refuses, with the reason)
    scratch = x_out.new_empty((nbytes // 4,)) if nbytes > 0 else None
    _call_packed("block_norm_backward",
                 _BLOCK_BACKWARD_ARGS.pack(*fields, *inputs, *tdx, *tdy, ppre, ppost, pgate, dgate_st,
                                           scratch.data_ptr() if nbytes > 0 else 0, max(0, nbytes)), device)
    return dx, dy, dpre_weight, dpost_weight, dgate
