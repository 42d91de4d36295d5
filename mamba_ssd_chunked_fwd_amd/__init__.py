"""Mamba-2 SSD chunked forward on AMD Instinct MI355X (gfx950).

A thin Python binding over libssd's C ABI (``include/ssd.h``,
``include/ssd_block.h`` and ``include/ssd_selective.h``).  Every step of
the computation runs in the library's HIP kernels; this module only checks
tensor shapes/dtypes, builds the dims struct and passes device pointers and
the current HIP stream.  PyTorch supplies device memory and streams.

Entry points (same names as the C ABI):
  ssd_chunk_cumsum, ssd_fwd_pass_state, ssd_chunk_state, ssd_state_passing,
  ssd_compute_out, ssd_state_and_out, ssd_forward, ssd_forward_noalloc,
  ssd_decode_step, ssd_causal_conv1d, ssd_gdn_chunk_fwd_h, ssd_gdn_chunk_fwd_o,
  ssd_linattn_fwd, ssd_linattn_bwd, ssd_linattn_step, ssd_add_norm_fwd,
  ssd_add_norm_bwd, ssd_gated_norm_fwd, ssd_gated_norm_bwd,
  ssd_short_conv_fwd, ssd_short_conv_bwd, ssd_short_conv_step,
  ssd_selective_scan_fwd, ssd_selective_scan_bwd, ssd_selective_scan_step,
  ssd_add_norm_quant_fwd
and the allocating convenience wrappers ``forward``, ``linattn``,
``linattn_backward``, ``add_norm``, ``add_norm_backward``, ``gated_norm``,
``gated_norm_backward``, ``short_conv``, ``short_conv_backward``,
``selective_scan``, ``selective_scan_backward`` and ``add_norm_quant``.

Importing fails loudly (ImportError) when libssd.so has not been built:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssd.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "ssd.h")
BLOCK_HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "ssd_block.h")
SELECTIVE_HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "ssd_selective.h")

SSD_OK = 0
SSD_ERR_INVALID_ARGUMENT = 1
SSD_ERR_UNSUPPORTED = 2
SSD_ERR_WORKSPACE = 3
SSD_ERR_HIP = 4
SSD_F32 = 0
SSD_BF16 = 1
SSD_GATES = {"silu": 0, "sigmoid": 1}
SSD_CONV_ACTS = {None: 0, "silu": 1}
SSD_CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}


class SsdDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk_size", ctypes.c_int64)]


class GdnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("dk", ctypes.c_int64),
                ("dv", ctypes.c_int64), ("chunk_size", ctypes.c_int64)]


class LinattnDims(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("nseq", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64)]


class GatedNormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("group", ctypes.c_int64), ("weight_dim", ctypes.c_int64)]


class ShortConvDims(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("nseq", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("width", ctypes.c_int64),
                ("x_stride", ctypes.c_int64)]


class SelectiveScanDims(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("nseq", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("ngroups", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64)]


class SsdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libssd.so not found at {LIB_PATH}; build it with "
            "`python mamba_ssd_chunked_fwd_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    dims = ctypes.POINTER(SsdDims)
    lib.ssd_status_string.argtypes = [i]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_forward_workspace_bytes.argtypes = [dims]
    lib.ssd_forward_workspace_bytes.restype = sz
    lib.ssd_chunk_cumsum.argtypes = [vp, vp, vp, vp, dims, vp]
    lib.ssd_chunk_cumsum.restype = i
    lib.ssd_fwd_pass_state.argtypes = [vp] * 7 + [i, dims, vp]
    lib.ssd_fwd_pass_state.restype = i
    lib.ssd_chunk_state.argtypes = [vp] * 6 + [i, dims, vp]
    lib.ssd_chunk_state.restype = i
    lib.ssd_state_passing.argtypes = [vp] * 4 + [dims, vp]
    lib.ssd_state_passing.restype = i
    lib.ssd_compute_out.argtypes = [vp] * 8 + [i, i, dims, vp]
    lib.ssd_compute_out.restype = i
    lib.ssd_state_and_out.argtypes = [vp] * 10 + [i, i, dims, vp]
    lib.ssd_state_and_out.restype = i
    lib.ssd_forward.argtypes = [vp] * 11 + [sz, i, i, dims, vp]
    lib.ssd_forward.restype = i
    lib.ssd_forward_noalloc.argtypes = [vp] * 10 + [i, i, dims, vp]
    lib.ssd_forward_noalloc.restype = i
    lib.ssd_decode_step.argtypes = [vp] * 8 + [i, i, dims, vp]
    lib.ssd_decode_step.restype = i
    i64 = ctypes.c_int64
    gdims = ctypes.POINTER(GdnDims)
    lib.ssd_gdn_chunk_fwd_h.argtypes = [vp] * 8 + [i, i, gdims, vp]
    lib.ssd_gdn_chunk_fwd_h.restype = i
    lib.ssd_gdn_chunk_fwd_o.argtypes = [vp] * 6 + [ctypes.c_float, i, i, i, gdims, vp]
    lib.ssd_gdn_chunk_fwd_o.restype = i
    lib.ssd_causal_conv1d.argtypes = [vp] * 4 + [i64] * 4 + [i, i, vp]
    lib.ssd_causal_conv1d.restype = i
    f = ctypes.c_float
    ldims = ctypes.POINTER(LinattnDims)
    for name in ("ssd_linattn_fwd_workspace_bytes", "ssd_linattn_bwd_workspace_bytes"):
        getattr(lib, name).argtypes = [ldims, i]
        getattr(lib, name).restype = sz
    lib.ssd_linattn_fwd.argtypes = [vp] * 9 + [sz, f, i, ldims, vp]
    lib.ssd_linattn_fwd.restype = i
    lib.ssd_linattn_bwd.argtypes = [vp] * 13 + [sz, f, i, ldims, vp]
    lib.ssd_linattn_bwd.restype = i
    lib.ssd_linattn_step.argtypes = [vp] * 6 + [f, i, ldims, vp]
    lib.ssd_linattn_step.restype = i
    lib.ssd_add_norm_fwd.argtypes = [vp] * 6 + [i64, i64, f, i, i, vp]
    lib.ssd_add_norm_fwd.restype = i
    lib.ssd_add_norm_bwd_workspace_bytes.argtypes = [i64, i64]
    lib.ssd_add_norm_bwd_workspace_bytes.restype = sz
    lib.ssd_add_norm_bwd.argtypes = [vp] * 11 + [sz, i64, i64, f, i, i, vp]
    lib.ssd_add_norm_bwd.restype = i
    ndims = ctypes.POINTER(GatedNormDims)
    lib.ssd_gated_norm_fwd.argtypes = [vp] * 4 + [f, i, i, i, i, ndims, vp]
    lib.ssd_gated_norm_fwd.restype = i
    lib.ssd_gated_norm_bwd_workspace_bytes.argtypes = [ndims]
    lib.ssd_gated_norm_bwd_workspace_bytes.restype = sz
    lib.ssd_gated_norm_bwd.argtypes = [vp] * 8 + [sz, f, i, i, i, i, ndims, vp]
    lib.ssd_gated_norm_bwd.restype = i
    cdims, sdims = ctypes.POINTER(ShortConvDims), ctypes.POINTER(SelectiveScanDims)
    lib.ssd_short_conv_fwd.argtypes = [vp] * 7 + [i, i, cdims, vp]
    lib.ssd_short_conv_fwd.restype = i
    lib.ssd_short_conv_bwd_workspace_bytes.argtypes = [cdims]
    lib.ssd_short_conv_bwd_workspace_bytes.restype = sz
    lib.ssd_short_conv_bwd.argtypes = [vp] * 12 + [sz, i, i, cdims, vp]
    lib.ssd_short_conv_bwd.restype = i
    lib.ssd_short_conv_step.argtypes = [vp] * 5 + [i, i, cdims, vp]
    lib.ssd_short_conv_step.restype = i
    for name in ("ssd_selective_scan_fwd_workspace_bytes",
                 "ssd_selective_scan_bwd_workspace_bytes"):
        getattr(lib, name).argtypes = [sdims, i]
        getattr(lib, name).restype = sz
    lib.ssd_selective_scan_fwd.argtypes = [vp] * 13 + [sz, i, i, sdims, vp]
    lib.ssd_selective_scan_fwd.restype = i
    lib.ssd_selective_scan_bwd.argtypes = [vp] * 22 + [sz, i, i, sdims, vp]
    lib.ssd_selective_scan_bwd.restype = i
    lib.ssd_selective_scan_step.argtypes = [vp] * 10 + [i, i, sdims, vp]
    lib.ssd_selective_scan_step.restype = i
    lib.ssd_add_norm_quant_fwd.argtypes = [vp] * 7 + [i64, i64, i64, f, i, i, i, vp]
    lib.ssd_add_norm_quant_fwd.restype = i
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    """The loaded libssd handle."""
    return _lib


def header_functions(path: str = HEADER_PATH) -> list:
    """Names of the functions a header (by default include/ssd.h) declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*"
                      r"(ssd_[a-z0-9_]+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    return _lib.ssd_status_string(int(status)).decode()


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return SSD_F32
    if t == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"unsupported dtype {t}; expected float32 or bfloat16")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: Optional[torch.Tensor], name: str, shape, dtypes,
           device=None, optional=False) -> None:
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must start on a 16-byte boundary (a slice of a "
                         f"larger tensor may not; pass a copy)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"{tuple(shape)}")


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def make_dims(x: torch.Tensor, B: torch.Tensor, chunk_size: int) -> SsdDims:
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [batch, seqlen, nheads, headdim] and B "
                         "[batch, seqlen, ngroups, dstate]")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return SsdDims(b, L, H, P, N, G, int(chunk_size))


def nchunks(d: SsdDims) -> int:
    return -(-d.seqlen // d.chunk_size)


def workspace_bytes(d: SsdDims) -> int:
    return int(_lib.ssd_forward_workspace_bytes(ctypes.byref(d)))


def _raise(st: int, where: str) -> None:
    if st != SSD_OK:
        raise SsdError(st, where)


# ------------------------------------------------------------- C-ABI entries
def ssd_chunk_cumsum(dt: torch.Tensor, A: torch.Tensor, g: torch.Tensor,
                     dt_t: torch.Tensor, chunk_size: int) -> None:
    """Stage 1: g [b, H, L] = log2(e) * per-chunk inclusive cumsum of A dt,
    and dt_t [b, H, L], dt transposed to head-major."""
    if dt.dim() != 3:
        raise ValueError("dt must be [batch, seqlen, nheads]")
    b, L, H = dt.shape
    f32 = (torch.float32,)
    _check(dt, "dt", None, f32)
    _check(A, "A", (H,), f32, dt.device)
    _check(g, "g", (b, H, L), f32, dt.device)
    _check(dt_t, "dt_t", (b, H, L), f32, dt.device)
    # stage 1 reads only batch, seqlen, nheads and chunk_size
    d = SsdDims(b, L, H, 64, 64, 1, int(chunk_size))
    _raise(_lib.ssd_chunk_cumsum(_ptr(dt), _ptr(A), _ptr(g), _ptr(dt_t),
                                 ctypes.byref(d), _stream(dt.device)),
           "ssd_chunk_cumsum")


def ssd_fwd_pass_state(x: torch.Tensor, B: torch.Tensor, dt_t: torch.Tensor,
                       g: torch.Tensor, init_state: Optional[torch.Tensor],
                       states: torch.Tensor,
                       final_state: Optional[torch.Tensor],
                       chunk_size: int) -> None:
    """Stage 2: per-chunk starting states [b, H, nc, P, N] and the final state."""
    d = make_dims(x, B, chunk_size)
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    _check(B, "B", (d.batch, d.seqlen, d.ngroups, d.dstate), (x.dtype,), dev)
    _check(dt_t, "dt_t", (d.batch, d.nheads, d.seqlen), f32, dev)
    _check(g, "g", (d.batch, d.nheads, d.seqlen), f32, dev)
    st_shape = (d.batch, d.nheads, d.headdim, d.dstate)
    _check(init_state, "init_state", st_shape, f32, dev, optional=True)
    _check(states, "states", (d.batch, d.nheads, nchunks(d), d.headdim,
                              d.dstate), f32, dev)
    _check(final_state, "final_state", st_shape, f32, dev, optional=True)
    _raise(_lib.ssd_fwd_pass_state(
        _ptr(x), _ptr(B), _ptr(dt_t), _ptr(g), _ptr(init_state), _ptr(states),
        _ptr(final_state), _dtype_code(x.dtype), ctypes.byref(d),
        _stream(dev)), "ssd_fwd_pass_state")


def ssd_chunk_state(x: torch.Tensor, B: torch.Tensor, dt_t: torch.Tensor,
                    g: torch.Tensor, states: torch.Tensor,
                    final_state: Optional[torch.Tensor], chunk_size: int) -> None:
    """Every chunk's zero-state contribution P_c into states[:, :, c+1]
    (P_{nc-1} into final_state); states[:, :, 0] is left as it is."""
    d = make_dims(x, B, chunk_size)
    dev = x.device
    b, L, H, P, N, nc = d.batch, d.seqlen, d.nheads, d.headdim, d.dstate, nchunks(d)
    f32 = (torch.float32,)
    _check(x, "x", None, (torch.float32, torch.bfloat16))
    _check(B, "B", (b, L, d.ngroups, N), (x.dtype,), dev)
    _check(dt_t, "dt_t", (b, H, L), f32, dev)
    _check(g, "g", (b, H, L), f32, dev)
    _check(states, "states", (b, H, nc, P, N), f32, dev)
    _check(final_state, "final_state", (b, H, P, N), f32, dev, optional=True)
    _raise(_lib.ssd_chunk_state(
        _ptr(x), _ptr(B), _ptr(dt_t), _ptr(g), _ptr(states), _ptr(final_state),
        _dtype_code(x.dtype), ctypes.byref(d), _stream(dev)), "ssd_chunk_state")


def ssd_state_passing(g: torch.Tensor, init_state: Optional[torch.Tensor],
                      states: torch.Tensor, final_state: Optional[torch.Tensor],
                      chunk_size: int) -> None:
    """In place: the chunk contributions left by ssd_chunk_state become the
    per-chunk starting states (and the final state)."""
    if states.dim() != 5:
        raise ValueError("states must be [batch, nheads, nchunks, headdim, dstate]")
    b, H, nc, P, N = states.shape
    L = g.shape[2] if g.dim() == 3 else -1
    dev = states.device
    f32 = (torch.float32,)
    _check(g, "g", (b, H, L), f32, dev)
    if -(-L // chunk_size) != nc:
        raise ValueError(f"states has {nc} chunks; g's {L} tokens make "
                         f"{-(-L // chunk_size)} chunks of {chunk_size}")
    _check(states, "states", None, f32, dev)
    _check(init_state, "init_state", (b, H, P, N), f32, dev, optional=True)
    _check(final_state, "final_state", (b, H, P, N), f32, dev, optional=True)
    d = SsdDims(b, L, H, P, N, 1, chunk_size)
    _raise(_lib.ssd_state_passing(
        _ptr(g), _ptr(init_state), _ptr(states), _ptr(final_state), ctypes.byref(d),
        _stream(dev)), "ssd_state_passing")


def ssd_compute_out(x: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                    dt_t: torch.Tensor, g: torch.Tensor, states: torch.Tensor,
                    D: torch.Tensor, y: torch.Tensor, chunk_size: int) -> None:
    """Stage 3: y [b, L, H, P] from the per-chunk starting states."""
    d = make_dims(x, B, chunk_size)
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    bc = (d.batch, d.seqlen, d.ngroups, d.dstate)
    _check(B, "B", bc, (x.dtype,), dev)
    _check(C, "C", bc, (x.dtype,), dev)
    _check(dt_t, "dt_t", (d.batch, d.nheads, d.seqlen), f32, dev)
    _check(g, "g", (d.batch, d.nheads, d.seqlen), f32, dev)
    _check(states, "states", (d.batch, d.nheads, nchunks(d), d.headdim,
                              d.dstate), f32, dev)
    _check(D, "D", (d.nheads,), f32, dev)
    _check(y, "y", tuple(x.shape), ins, dev)
    _raise(_lib.ssd_compute_out(
        _ptr(x), _ptr(B), _ptr(C), _ptr(dt_t), _ptr(g), _ptr(states), _ptr(D),
        _ptr(y), _dtype_code(x.dtype), _dtype_code(y.dtype), ctypes.byref(d),
        _stream(dev)), "ssd_compute_out")


def ssd_state_and_out(x: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                      dt_t: torch.Tensor, g: torch.Tensor, D: torch.Tensor,
                      init_state: Optional[torch.Tensor], y: torch.Tensor,
                      states: torch.Tensor, final_state: Optional[torch.Tensor],
                      chunk_size: int) -> None:
    """Stages 2 and 3 in one call (the fused single pass where it applies):
    states, final_state and y from stage 1's g and dt_t."""
    d = make_dims(x, B, chunk_size)
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    bc = (d.batch, d.seqlen, d.ngroups, d.dstate)
    _check(B, "B", bc, (x.dtype,), dev)
    _check(C, "C", bc, (x.dtype,), dev)
    _check(dt_t, "dt_t", (d.batch, d.nheads, d.seqlen), f32, dev)
    _check(g, "g", (d.batch, d.nheads, d.seqlen), f32, dev)
    _check(D, "D", (d.nheads,), f32, dev)
    st_shape = (d.batch, d.nheads, d.headdim, d.dstate)
    _check(init_state, "init_state", st_shape, f32, dev, optional=True)
    _check(y, "y", tuple(x.shape), ins, dev)
    _check(states, "states", (d.batch, d.nheads, nchunks(d), d.headdim,
                              d.dstate), f32, dev)
    _check(final_state, "final_state", st_shape, f32, dev, optional=True)
    _raise(_lib.ssd_state_and_out(
        _ptr(x), _ptr(B), _ptr(C), _ptr(dt_t), _ptr(g), _ptr(D), _ptr(init_state),
        _ptr(y), _ptr(states), _ptr(final_state), _dtype_code(x.dtype),
        _dtype_code(y.dtype), ctypes.byref(d), _stream(dev)), "ssd_state_and_out")


def ssd_forward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                B: torch.Tensor, C: torch.Tensor, D: torch.Tensor,
                init_state: Optional[torch.Tensor], y: torch.Tensor,
                states: torch.Tensor, final_state: Optional[torch.Tensor],
                workspace: torch.Tensor, chunk_size: int) -> None:
    """All three stages on the current stream; g and dt_t live in
    ``workspace`` (``workspace_bytes`` bytes)."""
    d = make_dims(x, B, chunk_size)
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    bc = (d.batch, d.seqlen, d.ngroups, d.dstate)
    _check(B, "B", bc, (x.dtype,), dev)
    _check(C, "C", bc, (x.dtype,), dev)
    _check(dt, "dt", (d.batch, d.seqlen, d.nheads), f32, dev)
    _check(A, "A", (d.nheads,), f32, dev)
    _check(D, "D", (d.nheads,), f32, dev)
    st_shape = (d.batch, d.nheads, d.headdim, d.dstate)
    _check(init_state, "init_state", st_shape, f32, dev, optional=True)
    _check(y, "y", tuple(x.shape), ins, dev)
    _check(states, "states", (d.batch, d.nheads, nchunks(d), d.headdim,
                              d.dstate), f32, dev)
    _check(final_state, "final_state", st_shape, f32, dev, optional=True)
    _check(workspace, "workspace", None, (torch.uint8, torch.float32), dev)
    nbytes = workspace.numel() * workspace.element_size()
    _raise(_lib.ssd_forward(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(init_state), _ptr(y), _ptr(states), _ptr(final_state),
        _ptr(workspace), nbytes, _dtype_code(x.dtype), _dtype_code(y.dtype),
        ctypes.byref(d), _stream(dev)), "ssd_forward")


NOALLOC_SCRATCH_BYTES = 32 << 20


def ssd_forward_noalloc(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                        B: torch.Tensor, C: torch.Tensor, D: torch.Tensor,
                        init_state: Optional[torch.Tensor], y: torch.Tensor,
                        states: torch.Tensor, final_state: Optional[torch.Tensor],
                        chunk_size: int) -> None:
    """``ssd_forward`` without a workspace: g and dt_t live in the library's
    per-GPU scratch array (NOALLOC_SCRATCH_BYTES), so the call allocates
    nothing.  Calls that overlap in time on one GPU race on that array."""
    d = make_dims(x, B, chunk_size)
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    bc = (d.batch, d.seqlen, d.ngroups, d.dstate)
    _check(B, "B", bc, (x.dtype,), dev)
    _check(C, "C", bc, (x.dtype,), dev)
    _check(dt, "dt", (d.batch, d.seqlen, d.nheads), f32, dev)
    _check(A, "A", (d.nheads,), f32, dev)
    _check(D, "D", (d.nheads,), f32, dev)
    st_shape = (d.batch, d.nheads, d.headdim, d.dstate)
    _check(init_state, "init_state", st_shape, f32, dev, optional=True)
    _check(y, "y", tuple(x.shape), ins, dev)
    _check(states, "states", (d.batch, d.nheads, nchunks(d), d.headdim,
                              d.dstate), f32, dev)
    _check(final_state, "final_state", st_shape, f32, dev, optional=True)
    _raise(_lib.ssd_forward_noalloc(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(init_state), _ptr(y), _ptr(states), _ptr(final_state),
        _dtype_code(x.dtype), _dtype_code(y.dtype), ctypes.byref(d), _stream(dev)),
        "ssd_forward_noalloc")


def ssd_decode_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                    B: torch.Tensor, C: torch.Tensor, D: torch.Tensor,
                    state: torch.Tensor, y: torch.Tensor) -> None:
    """One token for every (batch, head): ``state`` [b, H, P, N] fp32 is
    updated in place and ``y`` [b, H, P] written.  x [b, H, P], dt [b, H],
    B, C [b, G, N]."""
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [batch, nheads, headdim] and B "
                         "[batch, ngroups, dstate]")
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    d = SsdDims(b, 1, H, P, N, G, 64)
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    _check(B, "B", (b, G, N), (x.dtype,), dev)
    _check(C, "C", (b, G, N), (x.dtype,), dev)
    _check(dt, "dt", (b, H), f32, dev)
    _check(A, "A", (H,), f32, dev)
    _check(D, "D", (H,), f32, dev)
    _check(state, "state", (b, H, P, N), f32, dev)
    _check(y, "y", (b, H, P), ins, dev)
    _raise(_lib.ssd_decode_step(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(state),
        _ptr(y), _dtype_code(x.dtype), _dtype_code(y.dtype), ctypes.byref(d),
        _stream(dev)), "ssd_decode_step")


def ssd_gdn_chunk_fwd_h(k: torch.Tensor, w: torch.Tensor, u: torch.Tensor,
                        g: torch.Tensor, h0: Optional[torch.Tensor],
                        h: torch.Tensor, v_new: torch.Tensor,
                        final_state: Optional[torch.Tensor],
                        chunk_size: int = 64) -> None:
    """Gated DeltaNet state pass: k, w [b, L, H, K] and u [b, L, H, V] (bf16),
    g [b, L, H] fp32, h0 [b, H, K, V] fp32 or None; writes h [b, H, nt, K, V]
    fp32, v_new [b, L, H, V] (fp32 or bf16) and final_state (or None)."""
    if k.dim() != 4 or u.dim() != 4:
        raise ValueError("k must be [batch, seqlen, nheads, dk] and u "
                         "[batch, seqlen, nheads, dv]")
    b, L, H, K = k.shape
    V = u.shape[3]
    nt = -(-L // chunk_size)
    dev = k.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(k, "k", None, ins)
    _check(w, "w", (b, L, H, K), (k.dtype,), dev)
    _check(u, "u", (b, L, H, V), (k.dtype,), dev)
    _check(g, "g", (b, L, H), f32, dev)
    _check(h0, "h0", (b, H, K, V), f32, dev, optional=True)
    _check(h, "h", (b, H, nt, K, V), f32, dev)
    _check(v_new, "v_new", (b, L, H, V), ins, dev)
    _check(final_state, "final_state", (b, H, K, V), f32, dev, optional=True)
    d = GdnDims(b, L, H, K, V, chunk_size)
    _raise(_lib.ssd_gdn_chunk_fwd_h(
        _ptr(k), _ptr(w), _ptr(u), _ptr(g), _ptr(h0), _ptr(h), _ptr(v_new),
        _ptr(final_state), _dtype_code(k.dtype), _dtype_code(v_new.dtype),
        ctypes.byref(d), _stream(dev)), "ssd_gdn_chunk_fwd_h")


def ssd_gdn_chunk_fwd_o(q: torch.Tensor, k: torch.Tensor, v_new: torch.Tensor,
                        h: torch.Tensor, g: torch.Tensor, o: torch.Tensor,
                        scale: float = 1.0, chunk_size: int = 64) -> None:
    """Gated DeltaNet output: q, k [b, L, H, K] bf16; v_new [b, L, H, V] bf16;
    h [b, H, nt, K, V] fp32; g [b, L, H] fp32; writes o [b, L, H, V]
    (fp32 or bf16)."""
    if q.dim() != 4 or v_new.dim() != 4:
        raise ValueError("q must be [batch, seqlen, nheads, dk] and v_new "
                         "[batch, seqlen, nheads, dv]")
    b, L, H, K = q.shape
    V = v_new.shape[3]
    nt = -(-L // chunk_size)
    dev = q.device
    ins = (torch.float32, torch.bfloat16)
    _check(q, "q", None, ins)
    _check(k, "k", (b, L, H, K), (q.dtype,), dev)
    _check(v_new, "v_new", (b, L, H, V), ins, dev)
    _check(h, "h", (b, H, nt, K, V), (torch.float32,), dev)
    _check(g, "g", (b, L, H), (torch.float32,), dev)
    _check(o, "o", (b, L, H, V), ins, dev)
    d = GdnDims(b, L, H, K, V, chunk_size)
    _raise(_lib.ssd_gdn_chunk_fwd_o(
        _ptr(q), _ptr(k), _ptr(v_new), _ptr(h), _ptr(g), _ptr(o),
        ctypes.c_float(scale), _dtype_code(q.dtype), _dtype_code(v_new.dtype),
        _dtype_code(o.dtype), ctypes.byref(d), _stream(dev)), "ssd_gdn_chunk_fwd_o")


def ssd_causal_conv1d(x: torch.Tensor, weight: torch.Tensor,
                      bias: Optional[torch.Tensor], out: torch.Tensor) -> None:
    """Causal depthwise conv1d: x [batch, dim, seqlen] (fp32 or bf16),
    weight [dim, width] fp32, bias [dim] fp32 or None; writes ``out``
    [batch, dim, seqlen] (fp32 or bf16)."""
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [batch, dim, seqlen] and weight "
                         "[dim, width]")
    b, dim, L = x.shape
    W = weight.shape[1]
    dev = x.device
    ins = (torch.float32, torch.bfloat16)
    f32 = (torch.float32,)
    _check(x, "x", None, ins)
    _check(weight, "weight", (dim, W), f32, dev)
    _check(bias, "bias", (dim,), f32, dev, optional=True)
    _check(out, "out", (b, dim, L), ins, dev)
    _raise(_lib.ssd_causal_conv1d(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), b, dim, L, W,
        _dtype_code(x.dtype), _dtype_code(out.dtype), _stream(dev)),
        "ssd_causal_conv1d")


# --------------------------------------------------------- block operators
_FLOATS = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)


def _arg(t, name: str, shape, dtypes, device, optional: bool = False):
    """The address of a tensor that passes ``_check`` (None of an optional one).
    These calls take some microseconds: what is checked is looked at once here,
    and ``_check`` finds the words where something is wrong."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and \
            (shape is None or t.shape == shape) and t.is_cuda and t.is_contiguous():
        p = t.data_ptr()
        if p % 16 == 0:
            return p
    _check(t, name, shape, dtypes, device, optional)
    return None if t is None else t.data_ptr()


def _call(where: str, dev: torch.device, *args) -> None:
    """The entry point on the current stream of ``dev``, which need not be the
    current device."""
    f = getattr(_lib, where)
    # the handle that torch.cuda.current_stream(dev) wraps, without the wrapping
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch.cuda.current_device():
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st != SSD_OK:
        raise SsdError(st, where)


def _linattn_args(q, k, v, log_decay, init_state, cu_seqlens):
    """The dims of a linear attention call and the addresses of its inputs."""
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a tensor [batch, seqlen, heads, size]")
    b, L, G, K = q.shape
    H, V = v.shape[2:]
    dev, own = q.device, (q.dtype,)
    ptrs = [_arg(q, "q", None, _FLOATS, dev), _arg(k, "k", (b, L, G, K), own, dev),
            _arg(v, "v", (b, L, H, V), own, dev), _arg(log_decay, "log_decay", (H,), _F32, dev)]
    nseq = b
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 \
                or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a tensor [sequences + 1]")
        if b != 1:
            raise ValueError(f"packed sequences need a batch of 1, not {b}")
        nseq = cu_seqlens.numel() - 1
    cu = _arg(cu_seqlens, "cu_seqlens", None, (torch.int32,), dev, optional=True)
    ptrs += [_arg(init_state, "init_state", (nseq, H, K, V), _F32, dev, optional=True), cu]
    return LinattnDims(b * L, nseq, H, G, K, V), ptrs


def linattn_workspace_bytes(d: LinattnDims, dtype: torch.dtype, backward: bool = False) -> int:
    f = (_lib.ssd_linattn_bwd_workspace_bytes if backward
         else _lib.ssd_linattn_fwd_workspace_bytes)
    return int(f(ctypes.byref(d), _dtype_code(dtype)))


def _workspace(t: torch.Tensor, dev: torch.device):
    p = _arg(t, "workspace", None, (torch.uint8, torch.float32), dev)
    return p, t.numel() * t.element_size()


def _run_linattn_fwd(d, ins, v, o, final_state, workspace, scale) -> None:
    dev = v.device
    _call("ssd_linattn_fwd", dev, *ins, _arg(o, "o", v.shape, (v.dtype,), dev),
          _arg(final_state, "final_state", (d.nseq, d.nheads, d.dk, d.dv), _F32, dev, True),
          *workspace, d.dk ** -0.5 if scale is None else scale, _dtype_code(v.dtype), d)


def _run_linattn_bwd(d, ins, q, v, dout, dfinal, dq, dk, dv, dinit, workspace, scale) -> None:
    dev, own = v.device, (v.dtype,)
    state = (d.nseq, d.nheads, d.dk, d.dv)
    _call("ssd_linattn_bwd", dev, *ins, _arg(dout, "dout", v.shape, own, dev),
          _arg(dfinal, "dfinal", state, _F32, dev, True), _arg(dq, "dq", q.shape, own, dev),
          _arg(dk, "dk", q.shape, own, dev), _arg(dv, "dv", v.shape, own, dev),
          _arg(dinit, "dinit", state, _F32, dev, True), *workspace,
          d.dk ** -0.5 if scale is None else scale, _dtype_code(v.dtype), d)


def ssd_linattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    log_decay: torch.Tensor, init_state: Optional[torch.Tensor],
                    cu_seqlens: Optional[torch.Tensor], o: torch.Tensor,
                    final_state: Optional[torch.Tensor], workspace: torch.Tensor,
                    scale: Optional[float] = None) -> None:
    """Linear attention with a decay for each head: S_t = exp(log_decay) S_{t-1}
    + k_t v_t^T, o_t = scale q_t^T S_t.  q, k [b, L, G, K], v and o
    [b, L, H, V] (fp32 or bf16; H a multiple of G), log_decay [H] fp32; states
    [sequences, H, K, V] fp32 or None.  With cu_seqlens [sequences + 1] int32
    the sequences are packed in a batch of 1; else each batch row is one.
    ``workspace`` has linattn_workspace_bytes(dims, dtype) bytes.  scale None:
    K^-0.5."""
    d, ins = _linattn_args(q, k, v, log_decay, init_state, cu_seqlens)
    _run_linattn_fwd(d, ins, v, o, final_state, _workspace(workspace, v.device), scale)


def ssd_linattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    log_decay: torch.Tensor, init_state: Optional[torch.Tensor],
                    cu_seqlens: Optional[torch.Tensor], dout: torch.Tensor,
                    dfinal: Optional[torch.Tensor], dq: torch.Tensor, dk: torch.Tensor,
                    dv: torch.Tensor, dinit: Optional[torch.Tensor],
                    workspace: torch.Tensor, scale: Optional[float] = None) -> None:
    """Gradients of ``ssd_linattn_fwd`` for dout [b, L, H, V] and dfinal (or
    None) into dq, dk, dv and dinit (or None).  log_decay has none."""
    d, ins = _linattn_args(q, k, v, log_decay, init_state, cu_seqlens)
    _run_linattn_bwd(d, ins, q, v, dout, dfinal, dq, dk, dv, dinit,
                     _workspace(workspace, v.device), scale)


def ssd_linattn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     log_decay: torch.Tensor, state: torch.Tensor, o: torch.Tensor,
                     scale: Optional[float] = None) -> None:
    """One token of linear attention for every sequence: ``state`` [b, H, K, V]
    fp32 is updated in place and ``o`` [b, H, V] written.  q, k [b, G, K],
    v [b, H, V]."""
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a tensor [batch, heads, size]")
    b, G, K = q.shape
    H, V = v.shape[1:]
    dev, own = q.device, (q.dtype,)
    _call("ssd_linattn_step", dev, _arg(q, "q", None, _FLOATS, dev),
          _arg(k, "k", q.shape, own, dev), _arg(v, "v", (b, H, V), own, dev),
          _arg(log_decay, "log_decay", (H,), _F32, dev),
          _arg(state, "state", (b, H, K, V), _F32, dev), _arg(o, "o", v.shape, own, dev),
          K ** -0.5 if scale is None else scale, _dtype_code(q.dtype),
          LinattnDims(b, b, H, G, K, V))


def _rows(x: torch.Tensor, name: str) -> Tuple[int, int]:
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError(f"{name} must be a tensor [..., dim]")
    D = x.shape[-1]
    return (x.numel() // D if D else 0), D


def ssd_add_norm_fwd(x: torch.Tensor, residual: Optional[torch.Tensor],
                     res_scale: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                     y: torch.Tensor, residual_out: Optional[torch.Tensor],
                     eps: float = 1e-5) -> None:
    """h = residual + res_scale o x; residual_out = h; y = RMS norm of h, times
    weight.  x and y [..., dim] in one type, residual and residual_out in
    one (fp32 or bf16 each); res_scale and weight [dim] fp32.  residual,
    res_scale, weight and residual_out may be None."""
    rows, D = _rows(x, "x")
    dev, shape, own = x.device, x.shape, (x.dtype,)
    rdts = _FLOATS if residual is None else (residual.dtype,)
    rdt = next((t.dtype for t in (residual, residual_out) if t is not None), x.dtype)
    _call("ssd_add_norm_fwd", dev, _arg(x, "x", None, _FLOATS, dev),
          _arg(residual, "residual", shape, _FLOATS, dev, True),
          _arg(res_scale, "res_scale", (D,), _F32, dev, True),
          _arg(weight, "weight", (D,), _F32, dev, True), _arg(y, "y", shape, own, dev),
          _arg(residual_out, "residual_out", shape, rdts, dev, True), rows, D, eps,
          _dtype_code(x.dtype), _dtype_code(rdt))


def ssd_add_norm_bwd(x: torch.Tensor, residual: Optional[torch.Tensor],
                     res_scale: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                     dy: torch.Tensor, dresidual_out: Optional[torch.Tensor],
                     dx: torch.Tensor, dresidual: Optional[torch.Tensor],
                     dres_scale: Optional[torch.Tensor], dweight: Optional[torch.Tensor],
                     workspace: torch.Tensor, eps: float = 1e-5) -> None:
    """Gradients of ``ssd_add_norm_fwd`` from its inputs.  ``workspace`` has
    add_norm_workspace_bytes(rows, dim) bytes."""
    _run_add_norm_bwd(x, residual, res_scale, weight, dy, dresidual_out, dx, dresidual,
                      dres_scale, dweight, _workspace(workspace, x.device), eps)


def _run_add_norm_bwd(x, residual, res_scale, weight, dy, dresidual_out, dx, dresidual,
                      dres_scale, dweight, workspace, eps) -> None:
    rows, D = _rows(x, "x")
    dev, shape, own = x.device, x.shape, (x.dtype,)
    rdt = next((t.dtype for t in (residual, dresidual_out) if t is not None), x.dtype)
    rdts = _FLOATS if residual is None else (rdt,)
    _call("ssd_add_norm_bwd", dev, _arg(x, "x", None, _FLOATS, dev),
          _arg(residual, "residual", shape, _FLOATS, dev, True),
          _arg(res_scale, "res_scale", (D,), _F32, dev, True),
          _arg(weight, "weight", (D,), _F32, dev, True), _arg(dy, "dy", shape, own, dev),
          _arg(dresidual_out, "dresidual_out", shape, rdts, dev, True),
          _arg(dx, "dx", shape, own, dev),
          _arg(dresidual, "dresidual", shape, (rdt,), dev, True),
          _arg(dres_scale, "dres_scale", (D,), _F32, dev, True),
          _arg(dweight, "dweight", (D,), _F32, dev, True), *workspace, rows, D, eps,
          _dtype_code(x.dtype), _dtype_code(rdt))


def add_norm_workspace_bytes(rows: int, dim: int) -> int:
    return int(_lib.ssd_add_norm_bwd_workspace_bytes(rows, dim))


def _gate(gate: str) -> int:
    if gate not in SSD_GATES:
        raise ValueError(f"gate must be one of {sorted(SSD_GATES)}, not {gate!r}")
    return SSD_GATES[gate]


def _gated_args(x, z, weight, group):
    """The dims of a gated norm and the addresses of its inputs."""
    rows, D = _rows(x, "x")
    dev = x.device
    group = D if group is None else int(group)
    wdim = D
    if weight is not None:
        if not isinstance(weight, torch.Tensor) or weight.dim() != 1 \
                or weight.numel() not in (D, group):
            raise ValueError(f"weight must be a tensor [{D}] or [{group}]")
        wdim = weight.numel()
    return GatedNormDims(rows, D, group, wdim), [
        _arg(x, "x", None, _FLOATS, dev), _arg(z, "z", x.shape, _FLOATS, dev, True),
        _arg(weight, "weight", None, _F32, dev, True)]


def ssd_gated_norm_fwd(x: torch.Tensor, z: Optional[torch.Tensor],
                       weight: Optional[torch.Tensor], y: torch.Tensor, eps: float = 1e-5,
                       group: Optional[int] = None, gate: str = "silu",
                       gate_first: bool = False) -> None:
    """RMS norm of x [..., dim] over groups of channels (None: the whole row)
    with a gate act(z): y = norm(x o act(z)) o weight with gate_first, else
    y = norm(x) o weight o act(z).  z (or None: no gate) and y share a type,
    which x need not have; weight [dim] or [group] fp32 or None; gate "silu"
    or "sigmoid"."""
    d, ins = _gated_args(x, z, weight, group)
    dev = x.device
    _call("ssd_gated_norm_fwd", dev, *ins,
          _arg(y, "y", x.shape, _FLOATS if z is None else (z.dtype,), dev), eps, _gate(gate),
          int(gate_first), _dtype_code(x.dtype), _dtype_code(y.dtype), d)


def gated_norm_workspace_bytes(d: GatedNormDims) -> int:
    return int(_lib.ssd_gated_norm_bwd_workspace_bytes(ctypes.byref(d)))


def ssd_gated_norm_bwd(x: torch.Tensor, z: Optional[torch.Tensor],
                       weight: Optional[torch.Tensor], dy: torch.Tensor, dx: torch.Tensor,
                       dz: Optional[torch.Tensor], dweight: Optional[torch.Tensor],
                       workspace: torch.Tensor, eps: float = 1e-5,
                       group: Optional[int] = None, gate: str = "silu",
                       gate_first: bool = False) -> None:
    """Gradients of ``ssd_gated_norm_fwd`` from its inputs.  ``workspace`` has
    gated_norm_workspace_bytes(dims) bytes."""
    d, ins = _gated_args(x, z, weight, group)
    if isinstance(dweight, torch.Tensor) and weight is None:
        d.weight_dim = dweight.numel()
    _run_gated_norm_bwd(d, ins, x, z, dy, dx, dz, dweight, _workspace(workspace, x.device), eps,
                        gate, gate_first)


def _run_gated_norm_bwd(d, ins, x, z, dy, dx, dz, dweight, workspace, eps, gate,
                        gate_first) -> None:
    dev, shape = x.device, x.shape
    if (z is None) != (dz is None):
        raise ValueError("dz is given exactly when z is")
    _call("ssd_gated_norm_bwd", dev, *ins,
          _arg(dy, "dy", shape, _FLOATS if z is None else (z.dtype,), dev),
          _arg(dx, "dx", shape, (x.dtype,), dev), _arg(dz, "dz", shape, (dy.dtype,), dev, True),
          _arg(dweight, "dweight", (d.weight_dim,), _F32, dev, True), *workspace, eps,
          _gate(gate), int(gate_first), _dtype_code(x.dtype), _dtype_code(dy.dtype), d)


# ------------------------------------------- operators of a selective state space
def _rows_arg(t, name: str, shape, dtypes, device, size: int):
    """The address and the row stride (in elements) of a tensor whose rows (its last
    dimensions, ``shape`` being all of them) may be columns of a wider tensor.  It
    starts on a multiple of ``size`` bytes, and so does every row."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and \
            t.shape == shape and t.is_cuda:
        p = t.data_ptr()
        stride = 0 if t.is_contiguous() else _row_stride(name, t.shape, t.stride())
        if p % size == 0 and stride * t.element_size() % size == 0:
            return p, stride
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    stride = 0 if t.is_contiguous() else _row_stride(name, t.shape, t.stride())
    if stride * t.element_size() % size:
        raise ValueError(f"rows of {name} must be a multiple of {size} bytes apart (pass a copy)")
    if t.data_ptr() % size:
        raise ValueError(f"{name} must start on a {size}-byte boundary (pass a copy)")
    return t.data_ptr(), stride


@functools.lru_cache(maxsize=1024)
def _row_stride(name: str, shape, strides) -> int:
    """Elements between the rows of x [b, L, dim] or [b, dim], or of B [b, L, G, N] or
    [b, G, N]: rows contiguous, one distance between all of them."""
    lead = 2 if len(shape) == 4 or (len(shape) == 3 and name not in ("B", "C")) else 1
    inner = 1
    for n, s in zip(reversed(shape[lead:]), reversed(strides[lead:])):
        if n > 1 and s != inner:
            raise ValueError(f"{name}: the elements of a row must be contiguous (pass a copy)")
        inner *= n
    b, L = (1, shape[0]) if lead == 1 else shape[:2]
    if b * L == 1:
        return inner
    stride = strides[lead - 1] if L > 1 else strides[0]
    if stride < inner or (lead == 2 and b > 1 and L > 1 and strides[0] != L * stride):
        raise ValueError(f"{name}: rows must be one distance apart (pass a copy)")
    return stride


def _sequences(b: int, cu_seqlens, device):
    """The number of sequences and the address of cu_seqlens (None: each batch row is
    one sequence)."""
    if cu_seqlens is None:
        return b, None
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 \
            or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a tensor [sequences + 1]")
    if b != 1:
        raise ValueError(f"packed sequences need a batch of 1, not {b}")
    return cu_seqlens.numel() - 1, _arg(cu_seqlens, "cu_seqlens", None, (torch.int32,), device)


def _conv_act(activation: Optional[str]) -> int:
    if activation not in SSD_CONV_ACTS:
        raise ValueError(f"activation must be None or 'silu', not {activation!r}")
    return SSD_CONV_ACTS[activation]


def _conv_args(x, weight, bias, init_state, cu_seqlens):
    """The dims of a short convolution and the addresses of its inputs."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a tensor [batch, seqlen, dim]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [dim, width]")
    b, L, D = x.shape
    W, dev = weight.shape[1], x.device
    px, stride = _rows_arg(x, "x", x.shape, _FLOATS, dev, x.element_size())
    nseq, cu = _sequences(b, cu_seqlens, dev)
    return ShortConvDims(b * L, nseq, D, W, stride), [
        px, _arg(weight, "weight", (D, W), _F32, dev), _arg(bias, "bias", (D,), _F32, dev, True),
        _arg(init_state, "init_state", (nseq, W - 1, D), (x.dtype,), dev, True), cu]


def short_conv_workspace_bytes(d: ShortConvDims) -> int:
    return int(_lib.ssd_short_conv_bwd_workspace_bytes(ctypes.byref(d)))


def _run_conv_fwd(d, ins, x, y, final_state, activation) -> None:
    dev, own = x.device, (x.dtype,)
    _call("ssd_short_conv_fwd", dev, *ins, _arg(y, "y", x.shape, own, dev),
          _arg(final_state, "final_state", (d.nseq, d.width - 1, d.dim), own, dev, True),
          _conv_act(activation), _dtype_code(x.dtype), d)


def _run_conv_bwd(d, ins, x, dy, dfinal, dx, dweight, dbias, dinit, workspace,
                  activation) -> None:
    dev, own = x.device, (x.dtype,)
    state = (d.nseq, d.width - 1, d.dim)
    _call("ssd_short_conv_bwd", dev, *ins, _arg(dy, "dy", x.shape, own, dev),
          _arg(dfinal, "dfinal", state, own, dev, True), _arg(dx, "dx", x.shape, own, dev),
          _arg(dweight, "dweight", (d.dim, d.width), _F32, dev, True),
          _arg(dbias, "dbias", (d.dim,), _F32, dev, True),
          _arg(dinit, "dinit", state, own, dev, True), *workspace, _conv_act(activation),
          _dtype_code(x.dtype), d)


def ssd_short_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                       init_state: Optional[torch.Tensor], cu_seqlens: Optional[torch.Tensor],
                       y: torch.Tensor, final_state: Optional[torch.Tensor],
                       activation: Optional[str] = "silu") -> None:
    """The short causal convolution: y_t = act(bias + sum_k weight[:, k] x_{t-W+1+k}), the
    W - 1 rows before a sequence's first being init_state's (or zeros).  x, y [b, L, dim]
    (fp32 or bf16; rows of x may be columns of a wider tensor), weight [dim, W] and bias
    [dim] fp32 (bias may be None), states [sequences, W-1, dim] in x's type or None.
    With cu_seqlens [sequences + 1] int32 the sequences are packed in a batch of
    1; else each batch row is one.  activation "silu" or None."""
    d, ins = _conv_args(x, weight, bias, init_state, cu_seqlens)
    _run_conv_fwd(d, ins, x, y, final_state, activation)


def ssd_short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                       init_state: Optional[torch.Tensor], cu_seqlens: Optional[torch.Tensor],
                       dy: torch.Tensor, dfinal: Optional[torch.Tensor], dx: torch.Tensor,
                       dweight: Optional[torch.Tensor], dbias: Optional[torch.Tensor],
                       dinit: Optional[torch.Tensor], workspace: torch.Tensor,
                       activation: Optional[str] = "silu") -> None:
    """Gradients of ``ssd_short_conv_fwd`` from its inputs.  ``workspace`` has
    short_conv_workspace_bytes(dims) bytes."""
    d, ins = _conv_args(x, weight, bias, init_state, cu_seqlens)
    _run_conv_bwd(d, ins, x, dy, dfinal, dx, dweight, dbias, dinit,
                  _workspace(workspace, x.device), activation)


def ssd_short_conv_step(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                        state: torch.Tensor, y: torch.Tensor,
                        activation: Optional[str] = "silu") -> None:
    """One token of the short convolution for every sequence: ``state`` [b, W-1, dim] is
    updated in place and ``y`` [b, dim] written.  x [b, dim]."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [batch, dim]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [dim, width]")
    b, D = x.shape
    W, dev, own = weight.shape[1], x.device, (x.dtype,)
    px, stride = _rows_arg(x, "x", x.shape, _FLOATS, dev, x.element_size())
    _call("ssd_short_conv_step", dev, px, _arg(weight, "weight", (D, W), _F32, dev),
          _arg(bias, "bias", (D,), _F32, dev, True),
          _arg(state, "state", (b, W - 1, D), own, dev), _arg(y, "y", x.shape, own, dev),
          _conv_act(activation), _dtype_code(x.dtype), ShortConvDims(b, b, D, W, stride))


def _scan_args(x, dt, A, B, C, D, z, dt_bias, step: bool):
    """The dims of a selective scan (of a prompt's, all but nseq), and the addresses of its
    inputs."""
    lead = 1 if step else 2
    if not isinstance(x, torch.Tensor) or x.dim() != lead + 1:
        raise ValueError(f"x must be a tensor [batch, {'' if step else 'seqlen, '}dim]")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a tensor [dim, dstate]")
    if not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError(f"B must be a tensor [batch, {'' if step else 'seqlen, '}groups, dstate]")
    shape, dev, own, el = x.shape, x.device, (x.dtype,), x.element_size()
    dim, N, G = shape[-1], A.shape[1], B.shape[-2]
    bc = (*shape[:-1], G, N)
    px, xs = _rows_arg(x, "x", shape, _FLOATS, dev, el)
    pdt, dts = _rows_arg(dt, "dt", shape, own, dev, el)
    pB, bs = _rows_arg(B, "B", bc, own, dev, 4)
    pC, cs = _rows_arg(C, "C", bc, own, dev, 4)
    pz, zs = (None, 0) if z is None else _rows_arg(z, "z", shape, own, dev, el)
    rows = shape[0] if step else shape[0] * shape[1]
    return SelectiveScanDims(rows, rows, dim, N, G, xs, dts, zs, bs, cs), [
        px, pdt, _arg(A, "A", (dim, N), _F32, dev), pB, pC,
        None if D is None else _arg(D, "D", (dim,), _F32, dev), pz,
        None if dt_bias is None else _arg(dt_bias, "dt_bias", (dim,), _F32, dev)]


def _scan_prompt_args(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens):
    d, ins = _scan_args(x, dt, A, B, C, D, z, dt_bias, False)
    d.nseq, cu = _sequences(x.shape[0], cu_seqlens, x.device)
    ins += [_arg(init_state, "init_state", (d.nseq, d.dim, d.dstate), _F32, x.device, True), cu]
    return d, ins


def selective_scan_workspace_bytes(d: SelectiveScanDims, dtype: torch.dtype,
                                   backward: bool = False) -> int:
    f = (_lib.ssd_selective_scan_bwd_workspace_bytes if backward
         else _lib.ssd_selective_scan_fwd_workspace_bytes)
    return int(f(ctypes.byref(d), _dtype_code(dtype)))


def _run_scan_fwd(d, ins, x, y, final_state, workspace, softplus) -> None:
    dev = x.device
    _call("ssd_selective_scan_fwd", dev, *ins, _arg(y, "y", x.shape, (x.dtype,), dev),
          _arg(final_state, "final_state", (d.nseq, d.dim, d.dstate), _F32, dev, True),
          *workspace, int(softplus), _dtype_code(x.dtype), d)


def _run_scan_bwd(d, ins, x, dy, dfinal, grads, workspace, softplus) -> None:
    dev, own = x.device, (x.dtype,)
    dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit = grads
    if (ins[6] is None) != (dz is None):
        raise ValueError("dz is given exactly when z is")
    state, bc = (d.nseq, d.dim, d.dstate), x.shape[:-1] + (d.ngroups, d.dstate)
    _call("ssd_selective_scan_bwd", dev, *ins, _arg(dy, "dy", x.shape, own, dev),
          _arg(dfinal, "dfinal", state, _F32, dev, True), _arg(dx, "dx", x.shape, own, dev),
          _arg(ddt, "ddt", x.shape, own, dev), _arg(dA, "dA", (d.dim, d.dstate), _F32, dev),
          _arg(dB, "dB", bc, own, dev), _arg(dC, "dC", bc, own, dev),
          _arg(dD, "dD", (d.dim,), _F32, dev, True), _arg(dz, "dz", x.shape, own, dev, True),
          _arg(ddt_bias, "ddt_bias", (d.dim,), _F32, dev, True),
          _arg(dinit, "dinit", state, _F32, dev, True), *workspace, int(softplus),
          _dtype_code(x.dtype), d)


def ssd_selective_scan_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                           C: torch.Tensor, D: Optional[torch.Tensor],
                           z: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor],
                           init_state: Optional[torch.Tensor],
                           cu_seqlens: Optional[torch.Tensor], y: torch.Tensor,
                           final_state: Optional[torch.Tensor], workspace: torch.Tensor,
                           softplus: bool = True) -> None:
    """The selective scan: with delta = softplus(dt + dt_bias), per channel h_t =
    exp(delta_t A) h_{t-1} + delta_t x_t B_t and y_t = (C_t . h_t + D x_t) silu(z_t).
    x, dt, z, y [b, L, dim], B and C [b, L, G, N] (fp32 or bf16; rows of the inputs may be
    columns of wider tensors), A [dim, N], D and dt_bias [dim] fp32, states
    [sequences, dim, N] fp32; D, z, dt_bias and the states may be None.  Decays are meant
    to be at most 1 (delta A <= 0): where a product of larger ones over some tokens passes
    2^127 results may be NaN.  With
    cu_seqlens [sequences + 1] int32 the sequences are packed in a batch of 1; else each
    batch row is one.  ``workspace`` has selective_scan_workspace_bytes(dims, dtype)
    bytes."""
    d, ins = _scan_prompt_args(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens)
    _run_scan_fwd(d, ins, x, y, final_state, _workspace(workspace, x.device), softplus)


def ssd_selective_scan_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                           C: torch.Tensor, D: Optional[torch.Tensor],
                           z: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor],
                           init_state: Optional[torch.Tensor],
                           cu_seqlens: Optional[torch.Tensor], dy: torch.Tensor,
                           dfinal: Optional[torch.Tensor], dx: torch.Tensor, ddt: torch.Tensor,
                           dA: torch.Tensor, dB: torch.Tensor, dC: torch.Tensor,
                           dD: Optional[torch.Tensor], dz: Optional[torch.Tensor],
                           ddt_bias: Optional[torch.Tensor], dinit: Optional[torch.Tensor],
                           workspace: torch.Tensor, softplus: bool = True) -> None:
    """Gradients of ``ssd_selective_scan_fwd`` from its inputs, into contiguous tensors.
    ``workspace`` has selective_scan_workspace_bytes(dims, dtype, backward=True) bytes."""
    d, ins = _scan_prompt_args(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens)
    _run_scan_bwd(d, ins, x, dy, dfinal, (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit),
                  _workspace(workspace, x.device), softplus)


def ssd_selective_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                            B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor],
                            z: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor],
                            state: torch.Tensor, y: torch.Tensor,
                            softplus: bool = True) -> None:
    """One token of the selective scan for every sequence: ``state`` [b, dim, N] fp32 is
    updated in place and ``y`` [b, dim] written.  x, dt, z [b, dim], B, C [b, G, N]."""
    d, ins = _scan_args(x, dt, A, B, C, D, z, dt_bias, True)
    dev = x.device
    _call("ssd_selective_scan_step", dev, *ins,
          _arg(state, "state", (d.tokens, d.dim, d.dstate), _F32, dev),
          _arg(y, "y", x.shape, (x.dtype,), dev), int(softplus), _dtype_code(x.dtype), d)


def _quant_code(dtype: torch.dtype) -> int:
    if dtype not in SSD_CODES:
        raise ValueError(f"codes are torch.float8_e4m3fn or torch.int8, not {dtype}")
    return SSD_CODES[dtype]


def ssd_add_norm_quant_fwd(x: torch.Tensor, residual: Optional[torch.Tensor],
                           res_scale: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                           codes: torch.Tensor, scales: torch.Tensor,
                           residual_out: Optional[torch.Tensor], eps: float = 1e-5) -> None:
    """``ssd_add_norm_fwd`` with its output in 8 bits: ``codes`` [..., dim] (float8_e4m3fn
    or int8) and ``scales`` [..., dim / group] fp32, of which codes o scales stands for the
    normed row; the scales' last dimension gives the group (dim, or 16, 32, 64, 128 or
    256 channels)."""
    rows, D = _rows(x, "x")
    dev, shape = x.device, x.shape
    if not isinstance(codes, torch.Tensor) or not isinstance(scales, torch.Tensor):
        raise TypeError("codes and scales must be torch.Tensors")
    groups = scales.shape[-1] if scales.dim() else 0
    if not groups or D % groups:
        raise ValueError(f"scales must be a tensor [..., groups], groups a divisor of {D}")
    rdts = _FLOATS if residual is None else (residual.dtype,)
    rdt = next((t.dtype for t in (residual, residual_out) if t is not None), x.dtype)
    code = _quant_code(codes.dtype)
    _call("ssd_add_norm_quant_fwd", dev, _arg(x, "x", None, _FLOATS, dev),
          _arg(residual, "residual", shape, _FLOATS, dev, True),
          _arg(res_scale, "res_scale", (D,), _F32, dev, True),
          _arg(weight, "weight", (D,), _F32, dev, True),
          _arg(codes, "codes", shape, (codes.dtype,), dev),
          _arg(scales, "scales", shape[:-1] + (groups,), _F32, dev),
          _arg(residual_out, "residual_out", shape, rdts, dev, True), rows, D, D // groups, eps,
          code, _dtype_code(x.dtype), _dtype_code(rdt))


# ------------------------------------------------------------ convenience
def forward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
            B: torch.Tensor, C: torch.Tensor, D: torch.Tensor,
            init_state: Optional[torch.Tensor] = None, chunk_size: int = 64,
            y_dtype: torch.dtype = torch.float32
            ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Allocate outputs with torch.empty and run ``ssd_forward``.

    Returns (y [b, L, H, P] in y_dtype, states [b, H, nc, P, N] fp32,
    final_state [b, H, P, N] fp32).
    """
    d = make_dims(x, B, chunk_size)
    dev = x.device
    y = torch.empty(tuple(x.shape), dtype=y_dtype, device=dev)
    states = torch.empty((d.batch, d.nheads, nchunks(d), d.headdim, d.dstate),
                         dtype=torch.float32, device=dev)
    final = torch.empty((d.batch, d.nheads, d.headdim, d.dstate),
                        dtype=torch.float32, device=dev)
    # invalid or unsupported dims report 0 bytes; ssd_forward then returns the
    # precise status before touching the (minimal) workspace
    nbytes = max(workspace_bytes(d), 16)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ssd_forward(x, dt, A, B, C, D, init_state, y, states, final, ws,
                chunk_size)
    return y, states, final


def _scratch(n: int, dev: torch.device):
    """A workspace, its address and its bytes.  Invalid or unsupported dims report
    0 bytes; the call itself then returns the precise status before touching the
    (minimal) workspace."""
    n = max(n, 16)
    t = torch.empty(n, dtype=torch.uint8, device=dev)
    return t, (t.data_ptr(), n)


def _no_graph(where: str, **tensors) -> None:
    """Refuse tensors whose gradient a call would lose: the outputs carry no graph."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{where} records no graph, and {name} requires a gradient: call "
                                 f"it under torch.no_grad() and take gradients from "
                                 f"{where}_backward")


def linattn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
            init_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None,
            scale: Optional[float] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Allocate and run ``ssd_linattn_fwd``: (o, final_state).  Rows of o outside
    every packed sequence are not written.  No graph is recorded (gradients come
    from ``linattn_backward``): tensors that require one are refused outside
    torch.no_grad()."""
    _no_graph("linattn", q=q, k=k, v=v, log_decay=log_decay, init_state=init_state)
    d, ins = _linattn_args(q, k, v, log_decay, init_state, cu_seqlens)
    o = torch.empty_like(v)
    final = torch.empty((d.nseq, d.nheads, d.dk, d.dv), dtype=torch.float32, device=q.device)
    keep, ws = _scratch(linattn_workspace_bytes(d, q.dtype), q.device)
    _run_linattn_fwd(d, ins, v, o, final, ws, scale)
    return o, final


def linattn_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     log_decay: torch.Tensor, dout: torch.Tensor,
                     dfinal: Optional[torch.Tensor] = None,
                     init_state: Optional[torch.Tensor] = None,
                     cu_seqlens: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Allocate and run ``ssd_linattn_bwd``: (dq, dk, dv, dinit)."""
    d, ins = _linattn_args(q, k, v, log_decay, init_state, cu_seqlens)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dinit = torch.empty((d.nseq, d.nheads, d.dk, d.dv), dtype=torch.float32, device=q.device)
    keep, ws = _scratch(linattn_workspace_bytes(d, q.dtype, backward=True), q.device)
    _run_linattn_bwd(d, ins, q, v, dout, dfinal, dq, dk, dv, dinit, ws, scale)
    return dq, dk, dv, dinit


def add_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None,
             res_scale: Optional[torch.Tensor] = None,
             weight: Optional[torch.Tensor] = None,
             eps: float = 1e-5) -> Tuple[torch.Tensor, torch.Tensor]:
    """Allocate and run ``ssd_add_norm_fwd``: (y, residual_out).  No graph is recorded
    (gradients come from ``add_norm_backward``): tensors that require one are
    refused outside torch.no_grad()."""
    _no_graph("add_norm", x=x, residual=residual, res_scale=res_scale, weight=weight)
    y = torch.empty_like(x)
    out = torch.empty_like(x if residual is None else residual)
    ssd_add_norm_fwd(x, residual, res_scale, weight, y, out, eps)
    return y, out


def add_norm_backward(x: torch.Tensor, residual: Optional[torch.Tensor],
                      res_scale: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                      dy: torch.Tensor, dresidual_out: Optional[torch.Tensor] = None,
                      eps: float = 1e-5) -> Tuple[Optional[torch.Tensor], ...]:
    """Allocate and run ``ssd_add_norm_bwd``: (dx, dresidual, dres_scale,
    dweight), None for each of the last three whose input is None."""
    rows, D = _rows(x, "x")
    dx = torch.empty_like(x)
    dres, dscale, dw = (None if t is None else torch.empty_like(t)
                        for t in (residual, res_scale, weight))
    keep, ws = _scratch(add_norm_workspace_bytes(rows, D), x.device)
    _run_add_norm_bwd(x, residual, res_scale, weight, dy, dresidual_out, dx, dres, dscale, dw,
                      ws, eps)
    return dx, dres, dscale, dw


def gated_norm(x: torch.Tensor, z: Optional[torch.Tensor] = None,
               weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
               group: Optional[int] = None, gate: str = "silu",
               gate_first: bool = False) -> torch.Tensor:
    """Allocate and run ``ssd_gated_norm_fwd``: y, in z's type (x's without a
    gate).  No graph is recorded (gradients come from ``gated_norm_backward``):
    tensors that require one are refused outside torch.no_grad()."""
    _no_graph("gated_norm", x=x, z=z, weight=weight)
    y = torch.empty_like(x if z is None else z)
    ssd_gated_norm_fwd(x, z, weight, y, eps, group, gate, gate_first)
    return y


def gated_norm_backward(x: torch.Tensor, z: Optional[torch.Tensor],
                        weight: Optional[torch.Tensor], dy: torch.Tensor, eps: float = 1e-5,
                        group: Optional[int] = None, gate: str = "silu",
                        gate_first: bool = False) -> Tuple[Optional[torch.Tensor], ...]:
    """Allocate and run ``ssd_gated_norm_bwd``: (dx, dz, dweight), None for each
    of the last two whose input is None."""
    d, ins = _gated_args(x, z, weight, group)
    dx = torch.empty_like(x)
    dz, dw = (None if t is None else torch.empty_like(t) for t in (z, weight))
    keep, ws = _scratch(gated_norm_workspace_bytes(d), x.device)
    _run_gated_norm_bwd(d, ins, x, z, dy, dx, dz, dw, ws, eps, gate, gate_first)
    return dx, dz, dw


def short_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               init_state: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None,
               activation: Optional[str] = "silu") -> Tuple[torch.Tensor, torch.Tensor]:
    """Allocate and run ``ssd_short_conv_fwd``: (y, final_state).  Rows of y outside every
    packed sequence are not written.  No graph is recorded (gradients come from
    ``short_conv_backward``): tensors that require one are refused outside
    torch.no_grad()."""
    _no_graph("short_conv", x=x, weight=weight, bias=bias, init_state=init_state)
    d, ins = _conv_args(x, weight, bias, init_state, cu_seqlens)
    y, final = x.new_empty(x.shape), x.new_empty((d.nseq, d.width - 1, d.dim))
    _run_conv_fwd(d, ins, x, y, final, activation)
    return y, final


def short_conv_backward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                        dy: torch.Tensor, dfinal: Optional[torch.Tensor] = None,
                        init_state: Optional[torch.Tensor] = None,
                        cu_seqlens: Optional[torch.Tensor] = None,
                        activation: Optional[str] = "silu"
                        ) -> Tuple[Optional[torch.Tensor], ...]:
    """Allocate and run ``ssd_short_conv_bwd``: (dx, dweight, dbias, dinit), None for
    each of the last two whose input is None."""
    d, ins = _conv_args(x, weight, bias, init_state, cu_seqlens)
    dx, dw = x.new_empty(x.shape), torch.empty_like(weight)
    db, dinit = (None if t is None else torch.empty_like(t) for t in (bias, init_state))
    keep, ws = _scratch(short_conv_workspace_bytes(d), x.device)
    _run_conv_bwd(d, ins, x, dy, dfinal, dx, dw, db, dinit, ws, activation)
    return dx, dw, db, dinit


def selective_scan(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                   init_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None,
                   softplus: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """Allocate and run ``ssd_selective_scan_fwd``: (y, final_state).  Rows of y outside
    every packed sequence are not written.  No graph is recorded (gradients come from
    ``selective_scan_backward``): tensors that require one are refused outside
    torch.no_grad()."""
    _no_graph("selective_scan", x=x, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias,
              init_state=init_state)
    d, ins = _scan_prompt_args(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens)
    y, final = x.new_empty(x.shape), A.new_empty((d.nseq, d.dim, d.dstate))
    keep, ws = _scratch(selective_scan_workspace_bytes(d, x.dtype), x.device)
    _run_scan_fwd(d, ins, x, y, final, ws, softplus)
    return y, final


def selective_scan_backward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                            B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor],
                            z: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor],
                            dy: torch.Tensor, dfinal: Optional[torch.Tensor] = None,
                            init_state: Optional[torch.Tensor] = None,
                            cu_seqlens: Optional[torch.Tensor] = None, softplus: bool = True
                            ) -> Tuple[Optional[torch.Tensor], ...]:
    """Allocate and run ``ssd_selective_scan_bwd``: (dx, ddt, dA, dB, dC, dD, dz,
    ddt_bias, dinit), None for each of the last four whose input is None."""
    d, ins = _scan_prompt_args(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens)

    def like(t):
        return None if t is None else t.new_empty(t.shape)

    grads = [like(t) for t in (x, dt, A, B, C, D, z, dt_bias, init_state)]
    keep, ws = _scratch(selective_scan_workspace_bytes(d, x.dtype, backward=True), x.device)
    _run_scan_bwd(d, ins, x, dy, dfinal, grads, ws, softplus)
    return tuple(grads)


def add_norm_quant(x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                   res_scale: Optional[torch.Tensor] = None,
                   weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   dtype: torch.dtype = torch.float8_e4m3fn, group: Optional[int] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Allocate and run ``ssd_add_norm_quant_fwd``: (codes, scales, residual_out).  group
    None: one scale for each row.  The codes have no gradient: tensors that require one are
    refused outside torch.no_grad()."""
    if torch.is_grad_enabled():
        for name, t in (("x", x), ("residual", residual), ("res_scale", res_scale),
                        ("weight", weight)):
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"add_norm_quant has no gradient, and {name} requires one: call "
                                 f"it under torch.no_grad()")
    rows, D = _rows(x, "x")
    group = D if group is None else int(group)
    if group < 1 or D % group:
        raise ValueError(f"group must be a divisor of {D}, not {group}")
    codes = x.new_empty(x.shape, dtype=dtype)
    scales = x.new_empty(x.shape[:-1] + (D // group,), dtype=torch.float32)
    out = torch.empty_like(x if residual is None else residual)
    ssd_add_norm_quant_fwd(x, residual, res_scale, weight, codes, scales, out, eps)
    return codes, scales, out
