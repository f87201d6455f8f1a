"""Python binding of ``libssd_i8.so``: argument marshalling only.

Each function takes torch CUDA tensors, checks dtype / shape / contiguity, and passes their
device pointers to the C entry point of the same name (declared in ``include/ssd_i8.h``) on
the current torch stream.  All arithmetic runs in the library's CUDA kernels; if the library
is missing or fails to load, the calls raise -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
import warnings
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd_i8.so")

SSD_OK = 0
SSD_ERR_UNSUPPORTED = 2
STATUS_NAMES = {0: "SSD_OK", 1: "SSD_ERR_INVALID_ARG", 2: "SSD_ERR_UNSUPPORTED",
                3: "SSD_ERR_WORKSPACE", 4: "SSD_ERR_CUDA", 5: "SSD_ERR_TIMEOUT"}
OUT_DTYPES = {"f32": (0, torch.float32), "f16": (1, torch.float16), "i8": (2, torch.int8)}
OUT_HADAMARD = 16  # flag: y' = H y / 8 over headdim before the conversion (include/ssd_i8.h)
SCALES_PER_N = 32  # flag: B_scale / C_scale are [ngroups, dstate] (include/ssd_i8.h)

# names of every extern "C" symbol include/ssd_i8.h declares
EXPORTED = ("ssd_i8_abi_version", "ssd_status_string", "ssd_i8_chunk_scan_workspace_size",
            "ssd_i8_chunk_scan", "ssd_i8_state_update", "ssd_i8_chunk_cb",
            "ssd_i8_chunk_scan_noalloc", "ssd_i8_chunk_scan_status", "ssd_i8_debug_inject",
            "ssd_i8_chunk_scan_varlen_workspace_size", "ssd_i8_chunk_scan_varlen",
            "ssd_i8_state_quantize", "ssd_i8_state_update_q8", "ssd_i8_chunk_scan_noalloc_status",
            "ssd_i8_gated_scan", "ssd_i8_gated_scan_bwd", "ssd_i8_gated_scan_bwd_ckpt",
            "ssd_i8_gated_step", "ssd_i8_ckpt_pack", "ssd_i8_ckpt_unpack",
            "ssd_i8_gated_scan_workspace_size")

# the gated recurrence: element types, forms of the gate and of the input (include/ssd_i8.h)
IO_DTYPES = {"f32": (0, torch.float32), "f16": (1, torch.float16), "bf16": (3, torch.bfloat16)}
GATE_FORMS = {"log": 0, "logit": 1}
INPUT_FORMS = {"plain": 0, "complement": 16}
GATED_SPAN = 64  # tokens between the states that the forward saves for the backward
CKPT_BLOCK = 16  # tokens of one channel that share a checkpoint scale

# built-in scratch of ssd_i8_chunk_scan_noalloc (bytes); larger problems are refused
NOALLOC_SCRATCH_BYTES = 4 << 20

# kernels one ssd_i8_chunk_scan call launches (the fused persistent scan); the benchmark
# reports launches from it and a GPU test checks it against a profiler count
KERNELS_PER_CHUNK_SCAN = 1
KERNELS_PER_STATE_UPDATE = 1

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None
_tls = threading.local()  # device of the call being marshalled


class SSDError(RuntimeError):
    """A non-OK status returned by the library."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg}")
        self.status = status


def library() -> ctypes.CDLL:
    """Load ``libssd_i8.so`` (built by ``quantized_mamba_ssd_b200.build``) and declare types."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m quantized_mamba_ssd_b200.build` (no fallback exists)")
        lib = ctypes.CDLL(LIB_PATH)
        vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.ssd_i8_abi_version.restype = ci
        lib.ssd_i8_abi_version.argtypes = []
        lib.ssd_status_string.restype = ctypes.c_char_p
        lib.ssd_status_string.argtypes = [ci]
        lib.ssd_i8_chunk_scan_workspace_size.restype = sz
        lib.ssd_i8_chunk_scan_workspace_size.argtypes = [ci] * 7
        lib.ssd_i8_chunk_scan.restype = ci
        lib.ssd_i8_chunk_scan.argtypes = [vp] * 9 + [ci] * 7 + [vp, vp, vp, ci, cf, vp, sz, vp]
        lib.ssd_i8_state_update.restype = ci
        lib.ssd_i8_state_update.argtypes = [vp] * 10 + [ci] * 5 + [vp, ci, cf, vp]
        lib.ssd_i8_chunk_cb.restype = ci
        lib.ssd_i8_chunk_cb.argtypes = [vp, vp] + [ci] * 5 + [vp, vp]
        lib.ssd_i8_debug_inject.restype = ci
        lib.ssd_i8_debug_inject.argtypes = [ci, ctypes.c_longlong]
        lib.ssd_i8_chunk_scan_status.restype = ci
        lib.ssd_i8_chunk_scan_status.argtypes = [vp, vp]
        ll = ctypes.c_longlong
        lib.ssd_i8_chunk_scan_varlen_workspace_size.restype = sz
        lib.ssd_i8_chunk_scan_varlen_workspace_size.argtypes = [ci]
        lib.ssd_i8_chunk_scan_varlen.restype = ci
        lib.ssd_i8_chunk_scan_varlen.argtypes = ([vp, ll, vp, vp, ll, vp, ll] + [vp] * 5 +
                                                 [vp, ci, ll] + [ci] * 5 +
                                                 [vp, vp, vp, ci, cf, vp, sz, vp])
        lib.ssd_i8_state_quantize.restype = ci
        lib.ssd_i8_state_quantize.argtypes = [vp, vp, vp] + [ci] * 4 + [vp]
        lib.ssd_i8_state_update_q8.restype = ci
        lib.ssd_i8_state_update_q8.argtypes = [vp] * 11 + [ci] * 5 + [vp, ci, cf, vp]
        lib.ssd_i8_chunk_scan_noalloc.restype = ci
        lib.ssd_i8_chunk_scan_noalloc.argtypes = [vp] * 9 + [ci] * 7 + [vp, vp, vp, ci, cf, vp]
        lib.ssd_i8_chunk_scan_noalloc_status.restype = ci
        lib.ssd_i8_chunk_scan_noalloc_status.argtypes = [vp]
        rows = [vp, ll, ll]
        lib.ssd_i8_gated_scan.restype = ci
        lib.ssd_i8_gated_scan.argtypes = rows * 3 + [ci] * 3 + [vp, ci, ci, ci] + [vp] * 8 + [sz, vp]
        lib.ssd_i8_gated_scan_bwd.restype = ci
        lib.ssd_i8_gated_scan_bwd.argtypes = (rows * 5 + [ci] * 3 + [vp, ci, ci, ci] + [vp] * 5 +
                                              [sz, vp])
        lib.ssd_i8_gated_scan_bwd_ckpt.restype = ci
        lib.ssd_i8_gated_scan_bwd_ckpt.argtypes = (rows + [vp] * 4 + rows * 2 + [ci] * 3 +
                                                   [vp, ci, ci, ci] + [vp] * 5 + [sz, vp])
        lib.ssd_i8_gated_scan_workspace_size.restype = sz
        lib.ssd_i8_gated_scan_workspace_size.argtypes = [ci] * 4
        lib.ssd_i8_gated_step.restype = ci
        lib.ssd_i8_gated_step.argtypes = [vp] * 4 + [ci] * 4 + [vp]
        lib.ssd_i8_ckpt_pack.restype = ci
        lib.ssd_i8_ckpt_pack.argtypes = rows + [ci] * 4 + [vp] * 3
        lib.ssd_i8_ckpt_unpack.restype = ci
        lib.ssd_i8_ckpt_unpack.argtypes = [vp, vp] + [ci] * 4 + [vp, vp]
        _lib = lib
        return lib


def _check(fn: str, status: int) -> None:
    if status != SSD_OK:
        msg = library().ssd_status_string(status).decode()
        raise SSDError(fn, status, msg)


@contextlib.contextmanager
def _on_device_of(t: torch.Tensor):
    """Run one library call with ``t``'s GPU as the current device: the library launches on the
    current device, and every tensor of the call must live on that one."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError("the library's tensors must be CUDA tensors")
    prev = getattr(_tls, "device", None)
    _tls.device = t.device
    try:
        with torch.cuda.device(t.device):
            yield
    finally:
        _tls.device = prev


def _device_call(fn):
    """Decorator: the wrapped call marshals and launches on the GPU of its first tensor."""
    @functools.wraps(fn)
    def wrapper(first, *args, **kwargs):
        with _on_device_of(first):
            return fn(first, *args, **kwargs)
    return wrapper


def _ptr(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape=None) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = getattr(_tls, "device", None)
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr() if t.numel() else None


def _bc_scales(B_scale: torch.Tensor, C_scale: torch.Tensor, G: int, N: int) -> tuple:
    """Pointers of the B and C scales, [G] per group or [G, N] per group and dstate channel,
    and the y_dtype flag that says which."""
    per_n = isinstance(B_scale, torch.Tensor) and B_scale.dim() == 2
    shape = (G, N) if per_n else (G,)
    return (_ptr(B_scale, "B_scale", torch.float32, shape),
            _ptr(C_scale, "C_scale", torch.float32, shape),
            SCALES_PER_N if per_n else 0)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def ssd_i8_chunk_scan_workspace_size(batch: int, seqlen: int, nheads: int, headdim: int,
                                     dstate: int, ngroups: int, chunk_size: int) -> int:
    return int(library().ssd_i8_chunk_scan_workspace_size(batch, seqlen, nheads, headdim, dstate,
                                                          ngroups, chunk_size))


@_device_call
def ssd_i8_chunk_scan(x: torch.Tensor, B: torch.Tensor, C: torch.Tensor, dt: torch.Tensor,
                      A: torch.Tensor, D: torch.Tensor, x_scale: torch.Tensor,
                      B_scale: torch.Tensor, C_scale: torch.Tensor, chunk_size: int, *,
                      init_state: Optional[torch.Tensor] = None,
                      final_state: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None, y_dtype: str = "f16",
                      y_scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
                      stream=None, hadamard: bool = False) -> torch.Tensor:
    """Chunked int8 SSD scan (see ``ssd_i8_chunk_scan`` in include/ssd_i8.h).  ``hadamard``
    applies the output transform y' = H y / 8 over headdim (``SSD_OUT_HADAMARD``).

    x int8 [b,l,h,p]; B, C int8 [b,l,g,n]; dt f32 [b,l,h]; A, D, x_scale f32 [h];
    B_scale, C_scale f32 [g] (or [g, n]: per dstate channel, ``SSD_SCALES_PER_N``); optional
    init_state / final_state f32 [b,h,p,n]; returns y
    [b,l,h,p] of ``y_dtype`` ("f32", "f16" or "i8"; "i8" uses ``y_scale``).  ``workspace`` is
    a uint8 CUDA tensor of at least ``ssd_i8_chunk_scan_workspace_size`` bytes; one is
    allocated through torch when omitted.
    """
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,l,h,p] and B/C [b,l,g,n]")
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code, tdt = OUT_DTYPES[y_dtype]
    if y is None:
        y = torch.empty((bsz, L, H, P), dtype=tdt, device=x.device)
    need = ssd_i8_chunk_scan_workspace_size(bsz, L, H, P, N, G, chunk_size)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    pb, pc, flag = _bc_scales(B_scale, C_scale, G, N)
    args = [
        _ptr(x, "x", torch.int8, (bsz, L, H, P)),
        _ptr(B, "B", torch.int8, (bsz, L, G, N)),
        _ptr(C, "C", torch.int8, (bsz, L, G, N)),
        _ptr(dt, "dt", torch.float32, (bsz, L, H)),
        _ptr(A, "A", torch.float32, (H,)),
        _ptr(D, "D", torch.float32, (H,)),
        _ptr(x_scale, "x_scale", torch.float32, (H,)),
        pb, pc,
        bsz, L, H, P, N, G, int(chunk_size),
        _ptr(init_state, "init_state", torch.float32, (bsz, H, P, N)),
        _ptr(final_state, "final_state", torch.float32, (bsz, H, P, N)),
        _ptr(y, "y", tdt, (bsz, L, H, P)),
        code | (OUT_HADAMARD if hadamard else 0) | flag, float(y_scale),
        _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(),
        _stream(stream),
    ]
    _check("ssd_i8_chunk_scan", library().ssd_i8_chunk_scan(*args))
    return y


def _rows_ptr(t: torch.Tensor, name: str, dtype: torch.dtype, inner_shape) -> tuple:
    """Pointer and token stride (elements) of a [T, *inner_shape] view whose inner dims are
    contiguous (a column slice of a wider row-major buffer is accepted)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape[1:]) != tuple(inner_shape):
        raise ValueError(f"{name} must have shape [T, {', '.join(map(str, inner_shape))}], "
                         f"got {tuple(t.shape)}")
    inner = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.shape[d] > 1 and t.stride(d) != inner:
            raise ValueError(f"{name}: the dims after the token dim must be contiguous")
        inner *= t.shape[d]
    return (t.data_ptr() if t.numel() else None), (t.stride(0) if t.shape[0] > 1 else inner)


def ssd_i8_chunk_scan_varlen_workspace_size(nseq: int) -> int:
    return int(library().ssd_i8_chunk_scan_varlen_workspace_size(int(nseq)))


@_device_call
def ssd_i8_chunk_scan_varlen(x: torch.Tensor, B: torch.Tensor, C: torch.Tensor, dt: torch.Tensor,
                             A: torch.Tensor, D: torch.Tensor, x_scale: torch.Tensor,
                             B_scale: torch.Tensor, C_scale: torch.Tensor, cu_seqlens,
                             chunk_size: int, *, init_state: Optional[torch.Tensor] = None,
                             final_state: Optional[torch.Tensor] = None,
                             y: Optional[torch.Tensor] = None, y_dtype: str = "f16",
                             y_scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
                             stream=None, hadamard: bool = False) -> torch.Tensor:
    """Chunked int8 SSD scan over packed variable-length sequences (see
    ``ssd_i8_chunk_scan_varlen`` in include/ssd_i8.h).

    x int8 [T,h,p], B, C int8 [T,g,n], dt f32 [T,h]: token-major views whose inner dims are
    contiguous (column slices of a projection output are fine; B and C share a token stride);
    ``cu_seqlens``: host sequence of nseq + 1 token offsets; init_state / final_state f32
    [nseq,h,p,n]; returns y [T,h,p] of ``y_dtype``.
    """
    if x.dim() != 3 or B.dim() != 3 or C.dim() != 3 or dt.dim() != 2:
        raise ValueError("x must be [T,h,p], B/C [T,g,n] and dt [T,h]")
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    cu = [int(v) for v in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    nseq = len(cu) - 1
    if nseq < 0:
        raise ValueError("cu_seqlens needs at least one entry")
    code, tdt = OUT_DTYPES[y_dtype]
    if y is None:
        y = torch.empty((T, H, P), dtype=tdt, device=x.device)
    xp, xs = _rows_ptr(x, "x", torch.int8, (H, P))
    bp, bs = _rows_ptr(B, "B", torch.int8, (G, N))
    cp, cs = _rows_ptr(C, "C", torch.int8, (G, N))
    dp, ds = _rows_ptr(dt, "dt", torch.float32, (H,))
    if bs != cs:
        raise ValueError("B and C must have the same token stride")
    if B.shape[0] != T or C.shape[0] != T or dt.shape[0] != T:
        raise ValueError("x, B, C and dt must have the same number of tokens")
    need = ssd_i8_chunk_scan_varlen_workspace_size(nseq)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    cu_arr = (ctypes.c_int32 * len(cu))(*cu)
    pbs, pcs, flag = _bc_scales(B_scale, C_scale, G, N)
    args = [
        xp, xs, bp, cp, bs, dp, ds,
        _ptr(A, "A", torch.float32, (H,)),
        _ptr(D, "D", torch.float32, (H,)),
        _ptr(x_scale, "x_scale", torch.float32, (H,)),
        pbs, pcs,
        ctypes.cast(cu_arr, ctypes.c_void_p), nseq, T, H, P, N, G, int(chunk_size),
        _ptr(init_state, "init_state", torch.float32, (nseq, H, P, N)),
        _ptr(final_state, "final_state", torch.float32, (nseq, H, P, N)),
        _ptr(y, "y", tdt, (T, H, P)),
        code | (OUT_HADAMARD if hadamard else 0) | flag, float(y_scale),
        _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(),
        _stream(stream),
    ]
    _check("ssd_i8_chunk_scan_varlen", library().ssd_i8_chunk_scan_varlen(*args))
    return y


@_device_call
def ssd_i8_state_update(state: torch.Tensor, x: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        dt: torch.Tensor, A: torch.Tensor, D: torch.Tensor,
                        x_scale: torch.Tensor, B_scale: torch.Tensor, C_scale: torch.Tensor, *,
                        y: Optional[torch.Tensor] = None, y_dtype: str = "f16",
                        y_scale: float = 1.0, stream=None, hadamard: bool = False) -> torch.Tensor:
    """One decode step, state f32 [b,h,p,n] updated in place; x int8 [b,h,p]; B, C int8
    [b,g,n]; dt f32 [b,h].  Returns y [b,h,p] of ``y_dtype`` (``hadamard``: y' = H y / 8 over
    headdim, ``SSD_OUT_HADAMARD``)."""
    bsz, H, P, N = state.shape
    G = B.shape[1]
    code, tdt = OUT_DTYPES[y_dtype]
    if y is None:
        y = torch.empty((bsz, H, P), dtype=tdt, device=state.device)
    pb, pc, flag = _bc_scales(B_scale, C_scale, G, N)
    args = [
        _ptr(state, "state", torch.float32, (bsz, H, P, N)),
        _ptr(x, "x", torch.int8, (bsz, H, P)),
        _ptr(B, "B", torch.int8, (bsz, G, N)),
        _ptr(C, "C", torch.int8, (bsz, G, N)),
        _ptr(dt, "dt", torch.float32, (bsz, H)),
        _ptr(A, "A", torch.float32, (H,)),
        _ptr(D, "D", torch.float32, (H,)),
        _ptr(x_scale, "x_scale", torch.float32, (H,)),
        pb, pc,
        bsz, H, P, N, G,
        _ptr(y, "y", tdt, (bsz, H, P)),
        code | (OUT_HADAMARD if hadamard else 0) | flag, float(y_scale),
        _stream(stream),
    ]
    _check("ssd_i8_state_update", library().ssd_i8_state_update(*args))
    return y


@_device_call
def ssd_i8_state_quantize(state: torch.Tensor, state_q: Optional[torch.Tensor] = None,
                          state_scale: Optional[torch.Tensor] = None, stream=None):
    """fp32 state [b,h,p,n] -> (int8 codes [b,h,p,n], float32 scales [b,h]) with scale =
    max|h| / 127 per (batch, head) (see ``ssd_i8_state_quantize`` in include/ssd_i8.h)."""
    bsz, H, P, N = state.shape
    if state_q is None:
        state_q = torch.empty((bsz, H, P, N), dtype=torch.int8, device=state.device)
    if state_scale is None:
        state_scale = torch.empty((bsz, H), dtype=torch.float32, device=state.device)
    _check("ssd_i8_state_quantize", library().ssd_i8_state_quantize(
        _ptr(state, "state", torch.float32, (bsz, H, P, N)),
        _ptr(state_q, "state_q", torch.int8, (bsz, H, P, N)),
        _ptr(state_scale, "state_scale", torch.float32, (bsz, H)), bsz, H, P, N,
        _stream(stream)))
    return state_q, state_scale


@_device_call
def ssd_i8_state_update_q8(state_q: torch.Tensor, state_scale: torch.Tensor, x: torch.Tensor,
                           B: torch.Tensor, C: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                           D: torch.Tensor, x_scale: torch.Tensor, B_scale: torch.Tensor,
                           C_scale: torch.Tensor, *, y: Optional[torch.Tensor] = None,
                           y_dtype: str = "f16", y_scale: float = 1.0,
                           stream=None, hadamard: bool = False) -> torch.Tensor:
    """One decode step on the int8 cached state, in place (see ``ssd_i8_state_update_q8``).

    state_q int8 [b,h,p,n] and state_scale f32 [b,h] are updated; x int8 [b,h,p]; B, C int8
    [b,g,n]; dt f32 [b,h]; returns y [b,h,p] of ``y_dtype`` (``hadamard``: y' = H y / 8 over
    headdim)."""
    bsz, H, P, N = state_q.shape
    G = B.shape[1]
    code, tdt = OUT_DTYPES[y_dtype]
    if y is None:
        y = torch.empty((bsz, H, P), dtype=tdt, device=state_q.device)
    pb, pc, flag = _bc_scales(B_scale, C_scale, G, N)
    args = [
        _ptr(state_q, "state_q", torch.int8, (bsz, H, P, N)),
        _ptr(state_scale, "state_scale", torch.float32, (bsz, H)),
        _ptr(x, "x", torch.int8, (bsz, H, P)),
        _ptr(B, "B", torch.int8, (bsz, G, N)),
        _ptr(C, "C", torch.int8, (bsz, G, N)),
        _ptr(dt, "dt", torch.float32, (bsz, H)),
        _ptr(A, "A", torch.float32, (H,)),
        _ptr(D, "D", torch.float32, (H,)),
        _ptr(x_scale, "x_scale", torch.float32, (H,)),
        pb, pc,
        bsz, H, P, N, G,
        _ptr(y, "y", tdt, (bsz, H, P)),
        code | (OUT_HADAMARD if hadamard else 0) | flag, float(y_scale),
        _stream(stream),
    ]
    _check("ssd_i8_state_update_q8", library().ssd_i8_state_update_q8(*args))
    return y


@_device_call
def ssd_i8_chunk_cb(C: torch.Tensor, B: torch.Tensor, chunk_size: int, *,
                    cb: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ChunkBMM export: int32 [b, ceil(l/Q), g, Q, Q] = Cq Bq^T per chunk and group."""
    bsz, L, G, N = C.shape
    Q = int(chunk_size)
    nch = (L + Q - 1) // Q
    if cb is None:
        cb = torch.empty((bsz, nch, G, Q, Q), dtype=torch.int32, device=C.device)
    args = [
        _ptr(C, "C", torch.int8, (bsz, L, G, N)),
        _ptr(B, "B", torch.int8, (bsz, L, G, N)),
        bsz, L, G, N, Q,
        _ptr(cb, "cb", torch.int32, (bsz, nch, G, Q, Q)),
        _stream(stream),
    ]
    _check("ssd_i8_chunk_cb", library().ssd_i8_chunk_cb(*args))
    return cb


def ssd_i8_debug_inject(drop_publish_cta: int, wait_cycles: int) -> None:
    """Test hook: arm a one-shot hand-off fault for the next chunk scan (see include/ssd_i8.h)."""
    _check("ssd_i8_debug_inject", library().ssd_i8_debug_inject(int(drop_publish_cta), int(wait_cycles)))


@_device_call
def ssd_i8_chunk_scan_status(workspace: torch.Tensor, stream=None) -> None:
    """Raise SSDError (SSD_ERR_TIMEOUT) if a chunk scan that ran on ``workspace`` since the
    previous status query on it (with none, since its first call) reported a device-side wait
    that gave up; synchronises the stream."""
    _check("ssd_i8_chunk_scan_status",
           library().ssd_i8_chunk_scan_status(_ptr(workspace, "workspace", torch.uint8),
                                              _stream(stream)))


@_device_call
def ssd_i8_chunk_scan_noalloc(x: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                              dt: torch.Tensor, A: torch.Tensor, D: torch.Tensor,
                              x_scale: torch.Tensor, B_scale: torch.Tensor,
                              C_scale: torch.Tensor, chunk_size: int, *,
                              init_state: Optional[torch.Tensor] = None,
                              final_state: Optional[torch.Tensor] = None,
                              y: Optional[torch.Tensor] = None, y_dtype: str = "f16",
                              y_scale: float = 1.0, stream=None) -> torch.Tensor:
    """The chunk scan without a workspace, for callers that cannot allocate device memory:
    the library's built-in 4 MiB scratch (shared by all calls on a device) is used instead.
    Pass ``y`` to keep the call itself free of allocations; larger problems raise SSDError
    (SSD_ERR_WORKSPACE).  See ``ssd_i8_chunk_scan_noalloc`` in include/ssd_i8.h."""
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,l,h,p] and B/C [b,l,g,n]")
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code, tdt = OUT_DTYPES[y_dtype]
    if y is None:
        y = torch.empty((bsz, L, H, P), dtype=tdt, device=x.device)
    args = [
        _ptr(x, "x", torch.int8, (bsz, L, H, P)),
        _ptr(B, "B", torch.int8, (bsz, L, G, N)),
        _ptr(C, "C", torch.int8, (bsz, L, G, N)),
        _ptr(dt, "dt", torch.float32, (bsz, L, H)),
        _ptr(A, "A", torch.float32, (H,)),
        _ptr(D, "D", torch.float32, (H,)),
        _ptr(x_scale, "x_scale", torch.float32, (H,)),
        *_bc_scales(B_scale, C_scale, G, N)[:2],
        bsz, L, H, P, N, G, int(chunk_size),
        _ptr(init_state, "init_state", torch.float32, (bsz, H, P, N)),
        _ptr(final_state, "final_state", torch.float32, (bsz, H, P, N)),
        _ptr(y, "y", tdt, (bsz, L, H, P)),
        code | _bc_scales(B_scale, C_scale, G, N)[2], float(y_scale),
        _stream(stream),
    ]
    _check("ssd_i8_chunk_scan_noalloc", library().ssd_i8_chunk_scan_noalloc(*args))
    return y


def ssd_i8_chunk_scan_noalloc_status(stream=None) -> None:
    """Raise SSDError (SSD_ERR_TIMEOUT) if the last allocation-free chunk scan on the current
    device reported a device-side wait that gave up; synchronises the stream.  See
    ``ssd_i8_chunk_scan_noalloc_status`` in include/ssd_i8.h."""
    _check("ssd_i8_chunk_scan_noalloc_status",
           library().ssd_i8_chunk_scan_noalloc_status(_stream(stream)))


# ---------------------------------------------------------------------------------------
# gated linear recurrence and 8-bit activation checkpoints
# ---------------------------------------------------------------------------------------
_IO_CODES = {t: code for code, t in IO_DTYPES.values()}


def _raw_stream_of(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# handle of the current stream of GPU `dev`, without the Stream object around it (1.2 us of a
# 9 us decode step) where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream_of)
# the current GPU, likewise without the question whether CUDA is up: a CUDA tensor is at hand
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_said: set = set()  # the calls that have said so


def _not_recorded(name: str) -> None:
    """A call on tensors that require gradients, where torch records: says once per call that nothing is
    recorded.  (No error: the values are right, and a program may not want the gradients.)"""
    if name not in _said and torch.is_grad_enabled():
        _said.add(name)
        warnings.warn(f"{name} records no gradients, although its tensors require them: wrap it and its "
                      "backward call in a torch.autograd.Function, or call it under torch.no_grad()",
                      stacklevel=3)


class GatedCkpt(NamedTuple):
    """8-bit checkpoints of x and gate: int8 codes of the tensors' shape and uint8 exponents with
    ceil(l / 16) in the place of the token dim (``ssd_i8_gated_ckpt_empty`` allocates one)."""

    x_q: torch.Tensor
    x_e: torch.Tensor
    gate_q: torch.Tensor
    gate_e: torch.Tensor


def _gpu_of(first) -> int:
    """Index of the GPU that a call's first tensor lives on."""
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError("the library's tensors must be CUDA tensors")
    return first.get_device()


@contextlib.contextmanager
def _on(dev: int, stream):
    """``dev`` as the current device and, if given, ``stream`` (a torch stream or a raw handle) as
    the current stream: outputs that a call allocates then belong to the stream it runs on."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        with torch.cuda.stream(stream):
            yield


def _refuse(t, name: str, dtype: torch.dtype, shape: tuple, dev: int, what: str):
    """Why a tensor does not fit the call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}{what}")


def _flat(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple,
          dev: int) -> Optional[int]:
    """Pointer of a contiguous tensor on GPU ``dev`` (None passes)."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev, " must be contiguous")


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, dev: int) -> tuple:
    """Pointer, batch stride and token stride of [b, l, d] or [T, d] rows on GPU ``dev`` whose
    channels are contiguous."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev):
        st = t.stride()
        if st[-1] == 1 or shape[-1] <= 1 or not t.numel():
            return t.data_ptr(), (st[0] if len(st) == 3 else 0), st[-2]
    _refuse(t, name, dtype, shape, dev, ": the channels (last dim) must be contiguous")


def _out_rows(t: Optional[torch.Tensor], name: str, like: torch.Tensor, dev: int) -> tuple:
    """An output of the shape and dtype of ``like``, allocated where the caller gave none, and its
    pointer and strides."""
    if t is not None:
        return (t, *_rows(t, name, like.dtype, like.shape, dev))
    t, shape = _like(like), like.shape
    return t, t.data_ptr(), (shape[1] * shape[2] if len(shape) == 3 else 0), shape[-1]


_INT_MAX = 0x7fffffff


def _too_large(fn: str) -> None:
    """Refuses a size that the library, which takes C ints, would get cut by ctypes without a word."""
    _check(fn, SSD_ERR_UNSUPPORTED)


def _gated_shape(fn: str, t: torch.Tensor, name: str, cu_seqlens, dev: int) -> tuple:
    """(batch, tokens, channels, sequences, pointer of cu_seqlens, their count or 0) of a call on
    [b, l, d] rows, or on packed [T, d] rows with ``cu_seqlens``."""
    if cu_seqlens is None:
        if t.dim() != 3:
            raise ValueError(f"{name} must be [b,l,d], or [T,d] with cu_seqlens")
        b, l, d = t.shape
        if b > _INT_MAX or l > _INT_MAX or d > _INT_MAX:
            _too_large(fn)
        return b, l, d, b, None, 0
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T,d] with cu_seqlens")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be an int32 CUDA tensor of nseq + 1 token offsets")
    l, d = t.shape
    nseq = cu_seqlens.numel() - 1
    if l > _INT_MAX or d > _INT_MAX or nseq > _INT_MAX:
        _too_large(fn)
    return 1, l, d, nseq, _flat(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev), nseq


def _io_code(t: torch.Tensor, name: str) -> int:
    code = _IO_CODES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise TypeError(f"{name} must be a float32, float16 or bfloat16 tensor, got "
                        f"{getattr(t, 'dtype', type(t))}")
    return code


def _form(gate_form: str, input_form: str) -> int:
    try:
        return GATE_FORMS[gate_form] | INPUT_FORMS[input_form]
    except (KeyError, TypeError):
        raise ValueError(f"gate_form is one of {tuple(GATE_FORMS)}, input_form one of "
                         f"{tuple(INPUT_FORMS)}; got {gate_form!r}, {input_form!r}") from None


def _per(n: int, shape: tuple) -> tuple:
    """``shape`` [.., l, d] with ceil(l / n) in the place of l."""
    return (*shape[:-2], -(-shape[-2] // n), shape[-1])


def _like(x: torch.Tensor, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """A contiguous tensor of x's shape."""
    return (torch.empty_like(x, dtype=dtype) if x.is_contiguous()
            else x.new_empty(x.shape, dtype=dtype))


@functools.lru_cache(maxsize=4096)
def _gated_workspace_need(b: int, l: int, d: int, code: int, dev: int) -> int:
    """The library's answer for the current device ``dev``, which only depends on these numbers."""
    return library().ssd_i8_gated_scan_workspace_size(b, l, d, code)


def _gated_workspace(workspace, like: torch.Tensor, b: int, l: int, d: int, code: int,
                     dev: int) -> tuple:
    """The workspace of a scan (allocated where the caller gave none), its pointer and its size."""
    if workspace is None:
        need = _gated_workspace_need(b, l, d, code, dev)
        if not need:
            return None, None, 0
        workspace = like.new_empty(need, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
    return workspace, _flat(workspace, "workspace", torch.uint8, (n,), dev), n


def ssd_i8_gated_scan_workspace_size(batch: int, seqlen: int, channels: int, dtype: str) -> int:
    """Bytes of workspace of the gated scans, forward and backward ("f32", "f16" or "bf16"), on the
    current device."""
    if dtype not in IO_DTYPES:
        raise ValueError(f"dtype is one of {tuple(IO_DTYPES)}, got {dtype!r}")
    if not all(0 <= n <= _INT_MAX for n in (batch, seqlen, channels)):
        return 0  # as the library answers for sizes that it refuses
    return int(library().ssd_i8_gated_scan_workspace_size(batch, seqlen, channels,
                                                          IO_DTYPES[dtype][0]))


def _ckpt_ptrs(ckpt, shape: tuple, dev: int) -> tuple:
    if len(ckpt) != 4:
        raise ValueError("ckpt must hold x_q, x_e, gate_q and gate_e")
    e = _per(CKPT_BLOCK, shape)
    return (_flat(ckpt[0], "ckpt.x_q", torch.int8, shape, dev),
            _flat(ckpt[1], "ckpt.x_e", torch.uint8, e, dev),
            _flat(ckpt[2], "ckpt.gate_q", torch.int8, shape, dev),
            _flat(ckpt[3], "ckpt.gate_e", torch.uint8, e, dev))


def ssd_i8_gated_ckpt_empty(x: torch.Tensor) -> GatedCkpt:
    """Uninitialised 8-bit checkpoints for a gated scan of ``x`` ([b,l,d] or [T,d])."""
    if x.dim() not in (2, 3):
        raise ValueError("x must be [b,l,d] or [T,d]")
    q = _like(x, torch.int8)
    e = x.new_empty(_per(CKPT_BLOCK, x.shape), dtype=torch.uint8)
    return GatedCkpt(q, e, torch.empty_like(q), torch.empty_like(e))


def ssd_i8_gated_scan(x: torch.Tensor, gate: torch.Tensor,
                      cu_seqlens: Optional[torch.Tensor] = None, *, gate_form: str = "log",
                      input_form: str = "plain", init_state: Optional[torch.Tensor] = None,
                      final_state: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None,
                      span_states: Optional[torch.Tensor] = None,
                      ckpt: Optional[GatedCkpt] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gated linear recurrence h_t = a_t h_{t-1} + w_t x_t per channel, y_t = h_t (see
    ``ssd_i8_gated_scan`` in include/ssd_i8.h).

    x, gate [b,l,d], or packed [T,d] with ``cu_seqlens`` (int32 CUDA tensor of nseq + 1 token
    offsets), float32, float16 or bfloat16, channels contiguous and any batch and token stride.
    ``gate_form``: "log" (a = exp(gate)) or "logit" (a = sigmoid(gate)); ``input_form``: "plain"
    (w = 1) or "complement" (w = 1 - a).  init_state / final_state f32 [b,d] ([nseq,d] packed).
    For a backward pass: ``span_states`` f32 [b,ceil(l/64),d] ([ceil(T/64),d]) is written, and
    ``ckpt`` (``ssd_i8_gated_ckpt_empty``) receives x and gate in 8 bits.  ``workspace`` is a uint8
    CUDA tensor of at least ``ssd_i8_gated_scan_workspace_size`` bytes; one is allocated through
    torch when omitted.  Returns y, of x's shape and dtype; rows outside every packed sequence are
    left as they were.  Nothing is recorded for autograd (a warning says so where torch would record):
    a training program wraps this and the backward call in a ``torch.autograd.Function``."""
    dev = _gpu_of(x)
    if stream is not None or _current_device() != dev:
        with _on(dev, stream):
            return ssd_i8_gated_scan(x, gate, cu_seqlens, gate_form=gate_form,
                                     input_form=input_form, init_state=init_state,
                                     final_state=final_state, y=y, span_states=span_states,
                                     ckpt=ckpt, workspace=workspace)
    b, l, d, seqs, cu, nseq = _gated_shape("ssd_i8_gated_scan", x, "x", cu_seqlens, dev)
    code, dt, shape = _io_code(x, "x"), x.dtype, x.shape
    form = _form(gate_form, input_form)
    rows = (*_rows(x, "x", dt, shape, dev), *_rows(gate, "gate", dt, shape, dev))
    if x.requires_grad or gate.requires_grad or (init_state is not None and init_state.requires_grad):
        _not_recorded("ssd_i8_gated_scan")
    y, *y_rows = _out_rows(y, "y", x, dev)
    ws, pws, nws = _gated_workspace(workspace, x, b, l, d, code, dev)
    _check("ssd_i8_gated_scan", library().ssd_i8_gated_scan(
        *rows, *y_rows, b, l, d, cu, nseq, form, code,
        _flat(init_state, "init_state", torch.float32, (seqs, d), dev),
        _flat(final_state, "final_state", torch.float32, (seqs, d), dev),
        None if span_states is None else
        _flat(span_states, "span_states", torch.float32, _per(GATED_SPAN, shape), dev),
        *((None,) * 4 if ckpt is None else _ckpt_ptrs(ckpt, shape, dev)), pws, nws,
        _raw_stream(dev)))
    return y


def _gated_bwd(name, dy, inputs, span_states, cu_seqlens, gate_form, input_form, init_state,
               dfinal_state, dinit_state, dx, dgate, workspace, stream):
    dev = _gpu_of(dy)
    if stream is not None or _current_device() != dev:
        with _on(dev, stream):
            return _gated_bwd(name, dy, inputs, span_states, cu_seqlens, gate_form, input_form,
                              init_state, dfinal_state, dinit_state, dx, dgate, workspace, None)
    b, l, d, seqs, cu, nseq = _gated_shape(name, dy, "dy", cu_seqlens, dev)
    code, dt, shape = _io_code(dy, "dy"), dy.dtype, dy.shape
    form = _form(gate_form, input_form)
    if span_states is None:
        raise TypeError("span_states must be the tensor that the forward call wrote")
    rows = (*_rows(dy, "dy", dt, shape, dev), *inputs(dt, shape, dev))
    if dy.requires_grad:
        _not_recorded(name)
    dx, *dx_rows = _out_rows(dx, "dx", dy, dev)
    dgate, *dgate_rows = _out_rows(dgate, "dgate", dy, dev)
    ws, pws, nws = _gated_workspace(workspace, dy, b, l, d, code, dev)
    _check(name, getattr(library(), name)(
        *rows, *dx_rows, *dgate_rows, b, l, d, cu, nseq, form, code,
        _flat(init_state, "init_state", torch.float32, (seqs, d), dev),
        _flat(span_states, "span_states", torch.float32, _per(GATED_SPAN, shape), dev),
        _flat(dfinal_state, "dfinal_state", torch.float32, (seqs, d), dev),
        _flat(dinit_state, "dinit_state", torch.float32, (seqs, d), dev), pws, nws,
        _raw_stream(dev)))
    return dx, dgate


def ssd_i8_gated_scan_bwd(dy: torch.Tensor, x: torch.Tensor, gate: torch.Tensor,
                          span_states: torch.Tensor,
                          cu_seqlens: Optional[torch.Tensor] = None, *, gate_form: str = "log",
                          input_form: str = "plain", init_state: Optional[torch.Tensor] = None,
                          dfinal_state: Optional[torch.Tensor] = None,
                          dinit_state: Optional[torch.Tensor] = None,
                          dx: Optional[torch.Tensor] = None,
                          dgate: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """Gradients (dx, dgate) of ``ssd_i8_gated_scan`` for the gradient ``dy`` of its output.

    x, gate, cu_seqlens, the forms and init_state as in the forward call, span_states as it wrote
    them; dfinal_state f32 [b,d] ([nseq,d]) is the gradient of the final states, dinit_state
    receives that of the initial ones.  dy, x, gate, dx and dgate share shape and dtype; dx and
    dgate may be column slices of one wider buffer."""
    def inputs(dt, shape, dev):
        return (*_rows(x, "x", dt, shape, dev), *_rows(gate, "gate", dt, shape, dev))
    return _gated_bwd("ssd_i8_gated_scan_bwd", dy, inputs, span_states, cu_seqlens, gate_form,
                      input_form, init_state, dfinal_state, dinit_state, dx, dgate, workspace,
                      stream)


def ssd_i8_gated_scan_bwd_ckpt(dy: torch.Tensor, ckpt: GatedCkpt, span_states: torch.Tensor,
                               cu_seqlens: Optional[torch.Tensor] = None, *,
                               gate_form: str = "log", input_form: str = "plain",
                               init_state: Optional[torch.Tensor] = None,
                               dfinal_state: Optional[torch.Tensor] = None,
                               dinit_state: Optional[torch.Tensor] = None,
                               dx: Optional[torch.Tensor] = None,
                               dgate: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """``ssd_i8_gated_scan_bwd`` from the 8-bit checkpoints that the forward call wrote, in the
    place of x and gate."""
    def inputs(dt, shape, dev):
        return _ckpt_ptrs(ckpt, shape, dev)
    return _gated_bwd("ssd_i8_gated_scan_bwd_ckpt", dy, inputs, span_states, cu_seqlens,
                      gate_form, input_form, init_state, dfinal_state, dinit_state, dx, dgate,
                      workspace, stream)


def ssd_i8_gated_step(state: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, *,
                      gate_form: str = "log", input_form: str = "plain",
                      y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of ``ssd_i8_gated_scan`` for a decode batch: state f32 [b,d] updated in place;
    x, gate [b,d], contiguous.  Returns y [b,d] of x's dtype."""
    dev = _gpu_of(state)
    if stream is not None or _current_device() != dev:
        with _on(dev, stream):
            return ssd_i8_gated_step(state, x, gate, gate_form=gate_form, input_form=input_form,
                                     y=y)
    shape = state.shape
    if len(shape) != 2:
        raise ValueError("state must be [b,d]")
    b, d = shape
    if b > _INT_MAX or d > _INT_MAX:
        _too_large("ssd_i8_gated_step")
    code, dt, form = _io_code(x, "x"), x.dtype, _form(gate_form, input_form)
    ps = _flat(state, "state", torch.float32, shape, dev)
    px, pg = _flat(x, "x", dt, shape, dev), _flat(gate, "gate", dt, shape, dev)
    if x.requires_grad or gate.requires_grad or state.requires_grad:
        _not_recorded("ssd_i8_gated_step")
    if y is None:
        y = torch.empty_like(x)
        py = y.data_ptr()
    else:
        py = _flat(y, "y", dt, shape, dev)
    _check("ssd_i8_gated_step", library().ssd_i8_gated_step(
        ps, px, pg, py, b, d, form, code, _raw_stream(dev)))
    return y


def ssd_i8_ckpt_pack(x: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                     e: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """8-bit checkpoint of x [b,l,d] or [T,d] (float32, float16 or bfloat16, channels contiguous):
    (int8 codes of x's shape, uint8 exponents [b,ceil(l/16),d] or [ceil(T/16),d]); a value is
    code * 2^(exponent - 127) (see ``ssd_i8_ckpt_pack`` in include/ssd_i8.h)."""
    dev = _gpu_of(x)
    if stream is not None or _current_device() != dev:
        with _on(dev, stream):
            return ssd_i8_ckpt_pack(x, q=q, e=e)
    if x.dim() not in (2, 3):
        raise ValueError("x must be [b,l,d] or [T,d]")
    code, shape = _io_code(x, "x"), x.shape
    if max(shape) > _INT_MAX:
        _too_large("ssd_i8_ckpt_pack")
    rows, se = _rows(x, "x", x.dtype, shape, dev), _per(CKPT_BLOCK, shape)
    if x.requires_grad:
        _not_recorded("ssd_i8_ckpt_pack")
    if q is None:
        q = _like(x, torch.int8)
    if e is None:
        e = x.new_empty(se, dtype=torch.uint8)
    _check("ssd_i8_ckpt_pack", library().ssd_i8_ckpt_pack(
        *rows, shape[0] if len(shape) == 3 else 1, shape[-2], shape[-1], code,
        _flat(q, "q", torch.int8, shape, dev), _flat(e, "e", torch.uint8, se, dev),
        _raw_stream(dev)))
    return q, e


def ssd_i8_ckpt_unpack(q: torch.Tensor, e: torch.Tensor, *, dtype: str = "bf16",
                       x: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of an 8-bit checkpoint as ``dtype`` ("f32", "f16" or "bf16"), of q's shape."""
    dev = _gpu_of(q)
    if stream is not None or _current_device() != dev:
        with _on(dev, stream):
            return ssd_i8_ckpt_unpack(q, e, dtype=dtype, x=x)
    if q.dim() not in (2, 3):
        raise ValueError("q must be [b,l,d] or [T,d]")
    if dtype not in IO_DTYPES:
        raise ValueError(f"dtype is one of {tuple(IO_DTYPES)}, got {dtype!r}")
    (code, dt), shape = IO_DTYPES[dtype], q.shape
    if max(shape) > _INT_MAX:
        _too_large("ssd_i8_ckpt_unpack")
    pq = _flat(q, "q", torch.int8, shape, dev)
    pe = _flat(e, "e", torch.uint8, _per(CKPT_BLOCK, shape), dev)
    if x is None:
        x = _like(q, dt)
    _check("ssd_i8_ckpt_unpack", library().ssd_i8_ckpt_unpack(
        pq, pe, shape[0] if len(shape) == 3 else 1, shape[-2], shape[-1], code,
        _flat(x, "x", dt, shape, dev), _raw_stream(dev)))
    return x
