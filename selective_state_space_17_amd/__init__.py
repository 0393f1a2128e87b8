"""MI355X (gfx950) selective scan: thin Python binding of libmssm.so.

Every step of the computation runs in the library's HIP kernels; this module
only checks tensors, allocates outputs and workspace with torch (device memory
and streams are all torch is used for) and forwards raw pointers through the C
ABI declared in include/mssm.h.  There is no fallback path: if the library is
missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Any, NamedTuple, Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmssm.so")

MSSM_OK = 0
MSSM_ERR_INVALID_ARG = -1
MSSM_ERR_UNSUPPORTED = -2
MSSM_ERR_MISALIGNED = -3
MSSM_ERR_WORKSPACE = -4
MSSM_ERR_HIP = -5
MSSM_F32 = 0
MSSM_BF16 = 1


class ScanDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("split_seq", ctypes.c_int32),
                ("split_state", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class SSDDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class EmbeddingDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("scale", ctypes.c_float), ("io_dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("eps", ctypes.c_float),
                ("kind", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class CrossEntropyDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("ignore_id", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class Fp8Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("kind", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Fp8LinearDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("in_features", ctypes.c_int64), ("out_features", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("weight_kind", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


MSSM_LAYER_NORM = 0
MSSM_RMS_NORM = 1
MSSM_CROSS_ENTROPY_FINE_G = 2
MSSM_FP8_ROWS = 0
MSSM_FP8_SQUARE = 1
MSSM_E4M3 = 2


# every exported symbol and its ctypes signature (checked against include/mssm.h by the tests)
_P, _SZ, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
SIGNATURES = {
    "mssm_selective_scan_fwd": (_I, [ctypes.POINTER(ScanDesc)] + [_P] * 10 + [_P, _SZ, _P]),
    "mssm_selective_scan_workspace_size": (_SZ, [ctypes.POINTER(ScanDesc)]),
    "mssm_selective_scan_fwd_noalloc": (_I, [ctypes.POINTER(ScanDesc)] + [_P] * 10 + [_P]),
    "mssm_selective_scan_plan": (_I, [ctypes.POINTER(ScanDesc), ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(ctypes.c_int32)]),
    "mssm_ssd_fwd": (_I, [ctypes.POINTER(SSDDesc)] + [_P] * 10 + [_P, _SZ, _P]),
    "mssm_ssd_workspace_size": (_SZ, [ctypes.POINTER(SSDDesc)]),
    "mssm_ssd_plan": (_I, [ctypes.POINTER(SSDDesc), ctypes.POINTER(ctypes.c_int32)]),
    "mssm_ssd_mimo_plan": (_I, [ctypes.POINTER(SSDDesc), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    "mssm_ssd_mimo_fwd": (_I, [ctypes.POINTER(SSDDesc), ctypes.c_int32] + [_P] * 11 + [_P, _SZ, _P]),
    "mssm_ssd_mimo_state_update": (_I, [ctypes.POINTER(SSDDesc), ctypes.c_int32] + [_P] * 13),
    "mssm_ssd_trapezoidal_fwd": (_I, [ctypes.POINTER(SSDDesc)] + [_P] * 11 + [_P, _SZ, _P]),
    "mssm_selective_state_update": (_I, [ctypes.POINTER(ScanDesc)] + [_P] * 10),
    "mssm_ssd_state_update": (_I, [ctypes.POINTER(SSDDesc)] + [_P] * 10),
    "mssm_ssd_trapezoidal_state_update": (_I, [ctypes.POINTER(SSDDesc)] + [_P] * 13),
    "mssm_mamba3_siso_update": (_I, [ctypes.POINTER(SSDDesc)] + [_P] * 14),
    "mssm_selective_state_update_conv": (_I, [ctypes.POINTER(ScanDesc), ctypes.c_int32] + [_P] * 13),
    "mssm_selective_scan_conv_fwd": (_I, [ctypes.POINTER(ScanDesc), ctypes.c_int32] + [_P] * 13 + [_P, _SZ, _P]),
    "mssm_selective_scan_conv_workspace_size": (_SZ, [ctypes.POINTER(ScanDesc)]),
    "mssm_selective_scan_bwd": (_I, [ctypes.POINTER(ScanDesc)] + [_P] * 19 + [_P, _SZ, _P]),
    "mssm_selective_scan_fwd_ckpt": (_I, [ctypes.POINTER(ScanDesc)] + [_P] * 11 + [_P, _SZ, _P]),
    "mssm_selective_scan_fwd_ckpt_workspace_size": (_SZ, [ctypes.POINTER(ScanDesc)]),
    "mssm_selective_scan_checkpoint_size": (_SZ, [ctypes.POINTER(ScanDesc)]),
    "mssm_selective_scan_bwd_workspace_size": (_SZ, [ctypes.POINTER(ScanDesc)]),
    "mssm_embedding_fwd": (_I, [ctypes.POINTER(EmbeddingDesc)] + [_P] * 4),
    "mssm_embedding_bwd": (_I, [ctypes.POINTER(EmbeddingDesc)] + [_P] * 3 +
                           [ctypes.c_int32, ctypes.c_int32, _P, _SZ, _P]),
    "mssm_embedding_bwd_workspace_size": (_SZ, [ctypes.POINTER(EmbeddingDesc)]),
    "mssm_norm_fwd": (_I, [ctypes.POINTER(NormDesc)] + [_P] * 9),
    "mssm_norm_bwd": (_I, [ctypes.POINTER(NormDesc)] + [_P] * 11 + [_SZ, _P]),
    "mssm_norm_bwd_workspace_size": (_SZ, [ctypes.POINTER(NormDesc)]),
    "mssm_linear_cross_entropy_fwd": (_I, [ctypes.POINTER(CrossEntropyDesc)] + [_P] * 6 + [_SZ, _P]),
    "mssm_linear_cross_entropy_fwd_workspace_size": (_SZ, [ctypes.POINTER(CrossEntropyDesc)]),
    "mssm_linear_cross_entropy_bwd": (_I, [ctypes.POINTER(CrossEntropyDesc)] + [_P] * 8 +
                                      [ctypes.c_int32, ctypes.c_int32, _P, _SZ, _P]),
    "mssm_linear_cross_entropy_bwd_workspace_size": (_SZ, [ctypes.POINTER(CrossEntropyDesc)]),
    "mssm_fp8_quantize": (_I, [ctypes.POINTER(Fp8Desc)] + [_P] * 6),
    "mssm_fp8_transpose": (_I, [ctypes.POINTER(Fp8Desc)] + [_P] * 5),
    "mssm_fp8_dequantize": (_I, [ctypes.POINTER(Fp8Desc)] + [_P] * 4),
    "mssm_norm_fp8_fwd": (_I, [ctypes.POINTER(NormDesc)] + [_P] * 10),
    "mssm_fp8_linear_fwd": (_I, [ctypes.POINTER(Fp8LinearDesc)] + [_P] * 6 + [_SZ, _P]),
    "mssm_fp8_linear_fwd_workspace_size": (_SZ, [ctypes.POINTER(Fp8LinearDesc)]),
    "mssm_fp8_linear_bwd": (_I, [ctypes.POINTER(Fp8LinearDesc)] + [_P] * 7 +
                            [ctypes.c_int32, ctypes.c_int32, _P, _SZ, _P]),
    "mssm_fp8_linear_bwd_workspace_size": (_SZ, [ctypes.POINTER(Fp8LinearDesc)] + [ctypes.c_int32] * 3),
    "mssm_status_string": (ctypes.c_char_p, [_I]),
    "mssm_last_error_detail": (ctypes.c_char_p, []),
    "mssm_abi_version": (_I, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python selective_state_space_17_amd/build.py` "
                          "(or __graft_entry__.build()) first")
    # The library's HIP runtime dependency must resolve to the copy torch ships:
    # two HIP runtimes in one process leave the second without a device.  Load
    # torch first so libamdhip64 is already present when the library is opened.
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class MssmError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = lib.mssm_last_error_detail().decode() if status == MSSM_ERR_HIP else ""
        msg = f"{what}: {lib.mssm_status_string(status).decode()} ({status})"
        super().__init__(msg + (f": {detail}" if detail else ""))
        self.status = status


def abi_version() -> int:
    return lib.mssm_abi_version()


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_gpu(name, t, dtype, shape, cur):
    # Every check here runs on each call, so each uses the cheapest accessor (a decode step's
    # call is otherwise dominated by them): cur is the current device, looked up once per call,
    # get_device() is an int (-1 off the GPU), and a torch.Size compares equal to a tuple of
    # the same sizes.
    if t is None:
        return
    where = t.get_device()
    if where != cur:
        if where < 0:
            raise ValueError(f"{name} must be a GPU tensor")
        # the kernels run on the current device: a pointer into another GPU's memory would fault there
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur} "
                         "(use torch.cuda.device(...) around the call)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _io_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return MSSM_F32
    if dtype == torch.bfloat16:
        return MSSM_BF16
    raise TypeError(f"io dtype must be float32 or bfloat16, got {dtype}")


def _stream_handle(stream) -> int:
    torch = _torch()
    if stream is None:
        # the current stream of the current device (under graph capture: the capturing stream), as
        # its raw handle, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream belongs to {stream.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return stream.cuda_stream


def scan_desc(batch, seqlen, dim, dstate, io_dtype, split_seq=0, split_state=0) -> ScanDesc:
    return ScanDesc(batch, seqlen, dim, dstate, io_dtype, split_seq, split_state, 0)


def selective_scan_plan(batch: int, seqlen: int, dim: int, dstate: int, io_dtype: int = MSSM_BF16,
                        split_seq: int = 0, split_state: int = 0) -> Tuple[int, int]:
    """(sequence chunks, lanes per channel) the library picks for this problem."""
    d = scan_desc(batch, seqlen, dim, dstate, io_dtype, split_seq, split_state)
    k, g = ctypes.c_int32(0), ctypes.c_int32(0)
    st = lib.mssm_selective_scan_plan(ctypes.byref(d), ctypes.byref(k), ctypes.byref(g))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_scan_plan")
    return k.value, g.value


def selective_scan_workspace_size(batch, seqlen, dim, dstate, io_dtype=MSSM_BF16, split_seq=0, split_state=0) -> int:
    d = scan_desc(batch, seqlen, dim, dstate, io_dtype, split_seq, split_state)
    return lib.mssm_selective_scan_workspace_size(ctypes.byref(d))


def selective_scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None, return_final_state: bool = False,
                       split_seq: int = 0, split_state: int = 0, out=None, final_state=None, workspace=None,
                       stream=None):
    """Mamba-1 selective scan forward (mssm_selective_scan_fwd).

    x, delta, z: [batch, seqlen, dim]; B, C: [batch, seqlen, dstate] (float32 or bfloat16, all alike);
    A: [dim, dstate] float32; D: [dim] float32; h0: [batch, dim, dstate] float32.
    Returns out (and final_state [batch, dim, dstate] float32 when requested).
    """
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    bsz, L, dm = x.shape
    if A.dim() != 2 or A.shape[0] != dm:
        raise ValueError("A must be [dim, dstate]")
    N = A.shape[1]
    io = _io_code(x.dtype)
    cur = _torch().cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, dm)), ("delta", delta, (bsz, L, dm)), ("z", z, (bsz, L, dm)),
                           ("B", B, (bsz, L, N)), ("C", C, (bsz, L, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, dm, N), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, dm), cur)
    if return_final_state and final_state is None:
        final_state = torch.empty((bsz, dm, N), dtype=torch.float32, device=x.device)
    _check_gpu("final_state", final_state, torch.float32, (bsz, dm, N), cur)
    d = scan_desc(bsz, L, dm, N, io, split_seq, split_state)
    ws_bytes = lib.mssm_selective_scan_workspace_size(ctypes.byref(d))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    st = lib.mssm_selective_scan_fwd(ctypes.byref(d), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                     _ptr(z), _ptr(h0), _ptr(out), _ptr(final_state),
                                     _ptr(workspace) if ws_bytes else None,
                                     workspace.numel() if (ws_bytes and workspace is not None) else 0,
                                     _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_scan_fwd")
    return (out, final_state) if return_final_state else out


SCRATCH_BYTES = 32 << 20   # the per-device scratch mssm_selective_scan_fwd_noalloc keeps its chunk aggregates in


def selective_scan_fwd_noalloc(x, delta, A, B, C, D=None, z=None, h0=None, out=None, final_state=None,
                               split_seq: int = 0, split_state: int = 0, stream=None):
    """mssm_selective_scan_fwd_noalloc: the forward with no workspace (a split sequence keeps its chunk
    aggregates in the library's fixed per-device scratch).  ``out`` (and ``final_state``, when wanted)
    must be given, so that nothing is allocated here either; returns out."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    if out is None:
        raise ValueError("out must be given: this entry point allocates nothing")
    bsz, L, dm = x.shape
    if A.dim() != 2 or A.shape[0] != dm:
        raise ValueError("A must be [dim, dstate]")
    N = A.shape[1]
    io = _io_code(x.dtype)
    cur = torch.cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, dm)), ("delta", delta, (bsz, L, dm)), ("z", z, (bsz, L, dm)),
                           ("B", B, (bsz, L, N)), ("C", C, (bsz, L, N)), ("out", out, (bsz, L, dm))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, dm, N), cur)
    _check_gpu("final_state", final_state, torch.float32, (bsz, dm, N), cur)
    d = scan_desc(bsz, L, dm, N, io, split_seq, split_state)
    st = lib.mssm_selective_scan_fwd_noalloc(ctypes.byref(d), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                             _ptr(D), _ptr(z), _ptr(h0), _ptr(out), _ptr(final_state),
                                             _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_scan_fwd_noalloc")
    return out


def selective_scan_checkpoint_size(batch, seqlen, dim, dstate=16, io_dtype=MSSM_BF16) -> int:
    d = scan_desc(batch, seqlen, dim, dstate, io_dtype)
    return lib.mssm_selective_scan_checkpoint_size(ctypes.byref(d))


def selective_scan_fwd_ckpt(x, delta, A, B, C, D=None, z=None, h0=None, checkpoints=None,
                            return_final_state: bool = False, split_seq: int = 0, out=None, final_state=None,
                            workspace=None, stream=None):
    """Training-mode forward (mssm_selective_scan_fwd_ckpt): selective_scan_fwd that also stores the state
    entering every 16-step tile into ``checkpoints`` (allocated when None), for selective_scan_bwd.
    Returns (out, checkpoints) or (out, final_state, checkpoints)."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    bsz, L, dm = x.shape
    if A.dim() != 2 or A.shape[0] != dm:
        raise ValueError("A must be [dim, dstate]")
    N = A.shape[1]
    io = _io_code(x.dtype)
    cur = _torch().cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, dm)), ("delta", delta, (bsz, L, dm)), ("z", z, (bsz, L, dm)),
                           ("B", B, (bsz, L, N)), ("C", C, (bsz, L, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, dm, N), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, dm), cur)
    if return_final_state and final_state is None:
        final_state = torch.empty((bsz, dm, N), dtype=torch.float32, device=x.device)
    _check_gpu("final_state", final_state, torch.float32, (bsz, dm, N), cur)
    d = scan_desc(bsz, L, dm, N, io, split_seq, 16)
    ck_bytes = lib.mssm_selective_scan_checkpoint_size(ctypes.byref(d))
    if checkpoints is None:
        checkpoints = torch.empty(max(ck_bytes // 4, 1), dtype=torch.float32, device=x.device)
    elif not checkpoints.is_cuda or checkpoints.dtype != torch.float32 or checkpoints.numel() * 4 < ck_bytes:
        raise ValueError(f"checkpoints must be a float32 GPU tensor of at least {ck_bytes} bytes")
    ws_bytes = lib.mssm_selective_scan_fwd_ckpt_workspace_size(ctypes.byref(d))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    st = lib.mssm_selective_scan_fwd_ckpt(ctypes.byref(d), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                          _ptr(z), _ptr(h0), _ptr(out), _ptr(final_state), _ptr(checkpoints),
                                          _ptr(workspace) if ws_bytes else None,
                                          workspace.numel() if (ws_bytes and workspace is not None) else 0,
                                          _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_scan_fwd_ckpt")
    return (out, final_state, checkpoints) if return_final_state else (out, checkpoints)


def selective_scan_conv_workspace_size(batch, seqlen, dim, dstate, io_dtype=MSSM_BF16, split_seq=0) -> int:
    d = scan_desc(batch, seqlen, dim, dstate, io_dtype, split_seq, 16)
    return lib.mssm_selective_scan_conv_workspace_size(ctypes.byref(d))


def selective_scan_conv_fwd(xin, conv_w, conv_b, conv_init, delta, A, B, C, D=None, z=None, h0=None,
                            return_final_state: bool = False, split_seq: int = 0, out=None, final_state=None,
                            workspace=None, stream=None):
    """Selective scan with the short causal convolution + SiLU fused in front
    (mssm_selective_scan_conv_fwd): x = silu(conv_b + causal_conv(xin, conv_w)).

    xin, delta, z: [batch, seqlen, dim]; B, C: [batch, seqlen, dstate]; conv_w [dim, W] float32 (W 1..4);
    conv_b [dim] float32 or None; conv_init [batch, W-1, dim] in xin's dtype or None (read only).
    dstate 16 with rows of a multiple of 16 bytes runs on the fused block kernel; any other problem
    (dstate up to 256) on the recurrent kernel, token by token.
    """
    torch = _torch()
    if xin.dim() != 3:
        raise ValueError("xin must be [batch, seqlen, dim]")
    bsz, L, dm = xin.shape
    if A.dim() != 2 or A.shape[0] != dm:
        raise ValueError("A must be [dim, dstate]")
    if conv_w.dim() != 2 or conv_w.shape[0] != dm:
        raise ValueError("conv_w must be [dim, width]")
    N, W = A.shape[1], conv_w.shape[1]
    io = _io_code(xin.dtype)
    cur = _torch().cuda.current_device()
    for name, t, shape in (("xin", xin, (bsz, L, dm)), ("delta", delta, (bsz, L, dm)), ("z", z, (bsz, L, dm)),
                           ("B", B, (bsz, L, N)), ("C", C, (bsz, L, N)), ("conv_init", conv_init, (bsz, W - 1, dm))):
        _check_gpu(name, t, xin.dtype, shape, cur)
    _check_gpu("conv_w", conv_w, torch.float32, (dm, W), cur)
    _check_gpu("conv_b", conv_b, torch.float32, (dm,), cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, dm, N), cur)
    if out is None:
        out = torch.empty_like(xin)
    _check_gpu("out", out, xin.dtype, (bsz, L, dm), cur)
    if return_final_state and final_state is None:
        final_state = torch.empty((bsz, dm, N), dtype=torch.float32, device=xin.device)
    _check_gpu("final_state", final_state, torch.float32, (bsz, dm, N), cur)
    d = scan_desc(bsz, L, dm, N, io, split_seq, 16)
    ws_bytes = lib.mssm_selective_scan_conv_workspace_size(ctypes.byref(d))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=xin.device)
    st = lib.mssm_selective_scan_conv_fwd(ctypes.byref(d), W, _ptr(xin), _ptr(conv_w), _ptr(conv_b),
                                          _ptr(conv_init), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                          _ptr(h0), _ptr(out), _ptr(final_state),
                                          _ptr(workspace) if ws_bytes else None,
                                          workspace.numel() if (ws_bytes and workspace is not None) else 0,
                                          _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_scan_conv_fwd")
    return (out, final_state) if return_final_state else out


def selective_scan_bwd_workspace_size(batch, seqlen, dim, dstate, io_dtype=MSSM_BF16) -> int:
    d = scan_desc(batch, seqlen, dim, dstate, io_dtype)
    return lib.mssm_selective_scan_bwd_workspace_size(ctypes.byref(d))


def selective_scan_bwd(x, delta, A, B, C, D=None, z=None, h0=None, dout=None, dfinal=None, want_dh0: bool = True,
                       grads=None, checkpoints=None, workspace=None, stream=None):
    """Gradients of the Mamba-1 selective scan (mssm_selective_scan_bwd), for the loss
    sum(out * dout) + sum(final_state * dfinal).

    Inputs as in selective_scan_fwd; dout [batch, seqlen, dim] in the io dtype; dfinal
    [batch, dim, dstate] float32 or None.  Returns a dict: dx, ddelta, dz (io dtype, dz None without z),
    dB, dC [batch, seqlen, dstate] float32, dA [dim, dstate] float32, dD [dim] float32 (None without D),
    dh0 [batch, dim, dstate] float32 (None unless want_dh0).  ``grads`` may hold preallocated outputs
    (a dict with the same keys, as returned by an earlier call) to write into.  ``checkpoints``: the
    array selective_scan_fwd_ckpt filled for these inputs (dstate 16), which spares the kernel its own
    forward walk.
    """
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    bsz, L, dm = x.shape
    if A.dim() != 2 or A.shape[0] != dm:
        raise ValueError("A must be [dim, dstate]")
    N = A.shape[1]
    io = _io_code(x.dtype)
    if dout is None:
        raise ValueError("dout is required")
    cur = _torch().cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, dm)), ("delta", delta, (bsz, L, dm)), ("z", z, (bsz, L, dm)),
                           ("B", B, (bsz, L, N)), ("C", C, (bsz, L, N)), ("dout", dout, (bsz, L, dm))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, dm, N), cur)
    _check_gpu("dfinal", dfinal, torch.float32, (bsz, dm, N), cur)
    if checkpoints is not None:
        d0 = scan_desc(bsz, L, dm, N, io)
        need = lib.mssm_selective_scan_checkpoint_size(ctypes.byref(d0))
        if not checkpoints.is_cuda or checkpoints.dtype != torch.float32 or checkpoints.numel() * 4 < need:
            raise ValueError(f"checkpoints must be a float32 GPU tensor of at least {need} bytes")
    dev = x.device
    g = grads if grads is not None else {
        "dx": torch.empty_like(x), "ddelta": torch.empty_like(x),
        "dz": torch.empty_like(x) if z is not None else None,
        "dB": torch.empty((bsz, L, N), dtype=torch.float32, device=dev),
        "dC": torch.empty((bsz, L, N), dtype=torch.float32, device=dev),
        "dA": torch.empty((dm, N), dtype=torch.float32, device=dev),
        "dD": torch.empty((dm,), dtype=torch.float32, device=dev) if D is not None else None,
        "dh0": torch.empty((bsz, dm, N), dtype=torch.float32, device=dev) if want_dh0 else None,
    }
    if grads is not None:
        for name, dt, shape in (("dx", x.dtype, (bsz, L, dm)), ("ddelta", x.dtype, (bsz, L, dm)),
                                ("dz", x.dtype, (bsz, L, dm)), ("dB", torch.float32, (bsz, L, N)),
                                ("dC", torch.float32, (bsz, L, N)), ("dA", torch.float32, (dm, N)),
                                ("dD", torch.float32, (dm,)), ("dh0", torch.float32, (bsz, dm, N))):
            _check_gpu(name, g.get(name), dt, shape, cur)
    d = scan_desc(bsz, L, dm, N, io)
    ws_bytes = lib.mssm_selective_scan_bwd_workspace_size(ctypes.byref(d))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = lib.mssm_selective_scan_bwd(
        ctypes.byref(d), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(dout),
        _ptr(dfinal), _ptr(g["dx"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
        _ptr(g["dz"]), _ptr(g["dh0"]), _ptr(checkpoints), _ptr(workspace) if ws_bytes else None,
        workspace.numel() if (ws_bytes and workspace is not None) else 0, _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_scan_bwd")
    return g


def ssd_desc(batch, seqlen, nheads, headdim, dstate, ngroups, chunk=0, io_dtype=MSSM_BF16) -> SSDDesc:
    return SSDDesc(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, io_dtype, 0)


SSD_ROUTE_BLOCK = 0       # the matrix-core block kernel
SSD_ROUTE_RECURRENT = 1   # token by token through the update kernel


def ssd_plan(batch, seqlen, nheads, headdim, dstate, ngroups, chunk=0, io_dtype=MSSM_BF16) -> int:
    """Which kernel the multi-head forward runs this problem on (SSD_ROUTE_BLOCK or SSD_ROUTE_RECURRENT)."""
    d = ssd_desc(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, io_dtype)
    r = ctypes.c_int32(-1)
    st = lib.mssm_ssd_plan(ctypes.byref(d), ctypes.byref(r))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_ssd_plan")
    return r.value


def ssd_workspace_size(batch, seqlen, nheads, headdim, dstate, ngroups, chunk=0) -> int:
    d = ssd_desc(batch, seqlen, nheads, headdim, dstate, ngroups, chunk)
    return lib.mssm_ssd_workspace_size(ctypes.byref(d))


def ssd_fwd(x, delta, A, B, C, D=None, z=None, h0=None, chunk: int = 0, return_final_state: bool = False,
            out=None, final_state=None, workspace=None, stream=None):
    """Mamba-2 scalar-A multi-head forward (mssm_ssd_fwd).

    x, z: [batch, seqlen, nheads, headdim]; delta: [batch, seqlen, nheads]; B, C: [batch, seqlen,
    ngroups, dstate], all bfloat16 or all float32; A, D: [nheads] float32; h0: [batch, nheads, headdim,
    dstate] float32.  bfloat16 with headdim a multiple of 8 and dstate a multiple of 16 up to 256 runs
    on the matrix-core block kernel (above 128 states as two shares of the states, with a workspace);
    anything else (float32, other headdims, other dstate up to 256) on the recurrent kernel, token by
    token.
    """
    return _ssd_call("mssm_ssd_fwd", x, delta, None, A, B, C, D, z, h0, chunk, return_final_state, out,
                     final_state, workspace, stream)


def ssd_trapezoidal_fwd(x, delta, lam, A, B, C, D=None, z=None, h0=None, chunk: int = 0,
                        return_final_state: bool = False, out=None, final_state=None, workspace=None, stream=None):
    """Mamba-3 SISO recurrence, exponential-trapezoidal input rule (mssm_ssd_trapezoidal_fwd).

    As ``ssd_fwd`` plus lam: [batch, seqlen, nheads] in the I/O dtype, the weight of each step's own input (1 - lam
    goes to the previous step's input, carried through the step's decay).  lam = 1 gives ``ssd_fwd``.
    """
    return _ssd_call("mssm_ssd_trapezoidal_fwd", x, delta, lam, A, B, C, D, z, h0, chunk, return_final_state,
                     out, final_state, workspace, stream)


def ssd_mimo_plan(batch, seqlen, nheads, headdim, dstate, ngroups, rank, chunk=0, io_dtype=MSSM_BF16) -> int:
    """Which kernel mssm_ssd_mimo_fwd runs this problem on (SSD_ROUTE_BLOCK or SSD_ROUTE_RECURRENT)."""
    d = ssd_desc(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, io_dtype)
    r = ctypes.c_int32(-1)
    st = lib.mssm_ssd_mimo_plan(ctypes.byref(d), rank, ctypes.byref(r))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_ssd_mimo_plan")
    return r.value


def ssd_mimo_fwd(x, delta, lam, A, B, C, D=None, z=None, h0=None, chunk: int = 0, return_final_state: bool = False,
                 out=None, final_state=None, workspace=None, stream=None):
    """Mamba-3 MIMO (mssm_ssd_mimo_fwd): x, z [batch, seqlen, nheads, rank, headdim]; B, C [batch, seqlen,
    ngroups, rank, dstate]; delta, lam [batch, seqlen, nheads] (lam None: the Mamba-2 rule); A, D [nheads];
    h0 [batch, nheads, headdim, dstate].  Returns out (and the final state when asked)."""
    torch = _torch()
    if x.dim() != 5 or B.dim() != 5:
        raise ValueError("x must be [batch, seqlen, nheads, rank, headdim] and B [batch, seqlen, ngroups, rank, dstate]")
    bsz, L, H, R, P = x.shape
    G, N = B.shape[2], B.shape[4]
    io = _io_code(x.dtype)
    cur = torch.cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, H, R, P)), ("z", z, (bsz, L, H, R, P)), ("delta", delta, (bsz, L, H)),
                           ("lam", lam, (bsz, L, H)), ("B", B, (bsz, L, G, R, N)), ("C", C, (bsz, L, G, R, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (H,), cur)
    _check_gpu("D", D, torch.float32, (H,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, H, P, N), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, H, R, P), cur)
    if return_final_state and final_state is None:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=x.device)
    _check_gpu("final_state", final_state, torch.float32, (bsz, H, P, N), cur)
    d = ssd_desc(bsz, L, H, P, N, G, chunk, io)
    ws_bytes = lib.mssm_ssd_workspace_size(ctypes.byref(d))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    st = lib.mssm_ssd_mimo_fwd(ctypes.byref(d), R, _ptr(x), _ptr(delta), _ptr(lam), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(D), _ptr(z), _ptr(h0), _ptr(out), _ptr(final_state),
                               _ptr(workspace) if ws_bytes else None,
                               workspace.numel() if (ws_bytes and workspace is not None) else 0,
                               _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_ssd_mimo_fwd")
    return (out, final_state) if return_final_state else out


def ssd_mimo_state_update(state, x, delta, lam, A, B, C, D=None, z=None, x_prev=None, B_prev=None, out=None,
                          stream=None):
    """Advance a multi-head state by seqlen tokens in place under Mamba-3 MIMO (mssm_ssd_mimo_state_update).
    x, z [batch, seqlen, nheads, rank, headdim]; B, C [batch, seqlen, ngroups, rank, dstate]; lam None: the
    Mamba-2 rule; x_prev [batch, nheads, rank, headdim], B_prev [batch, ngroups, rank, dstate] (None: no
    previous token).  Returns out."""
    torch = _torch()
    if x.dim() != 5 or B.dim() != 5:
        raise ValueError("x must be [batch, seqlen, nheads, rank, headdim] and B [batch, seqlen, ngroups, rank, dstate]")
    bsz, L, H, R, P = x.shape
    G, N = B.shape[2], B.shape[4]
    io = _io_code(x.dtype)
    cur = torch.cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, H, R, P)), ("z", z, (bsz, L, H, R, P)), ("delta", delta, (bsz, L, H)),
                           ("lam", lam, (bsz, L, H)), ("B", B, (bsz, L, G, R, N)), ("C", C, (bsz, L, G, R, N)),
                           ("x_prev", x_prev, (bsz, H, R, P)), ("B_prev", B_prev, (bsz, G, R, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (H,), cur)
    _check_gpu("D", D, torch.float32, (H,), cur)
    _check_gpu("state", state, torch.float32, (bsz, H, P, N), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, H, R, P), cur)
    d = ssd_desc(bsz, L, H, P, N, G, 0, io)
    st = lib.mssm_ssd_mimo_state_update(ctypes.byref(d), R, _ptr(state), _ptr(x_prev), _ptr(B_prev), _ptr(x),
                                        _ptr(delta), _ptr(lam), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                        _ptr(out), _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_ssd_mimo_state_update")
    return out


def _ssd_call(fn, x, delta, lam, A, B, C, D, z, h0, chunk, return_final_state, out, final_state, workspace,
              stream):
    torch = _torch()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [batch, seqlen, nheads, headdim] and B [batch, seqlen, ngroups, dstate]")
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    io = _io_code(x.dtype)
    trap = fn == "mssm_ssd_trapezoidal_fwd"
    if trap and lam is None:
        raise ValueError("lam is required")
    cur = _torch().cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, H, P)), ("z", z, (bsz, L, H, P)), ("delta", delta, (bsz, L, H)),
                           ("lam", lam, (bsz, L, H)), ("B", B, (bsz, L, G, N)), ("C", C, (bsz, L, G, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (H,), cur)
    _check_gpu("D", D, torch.float32, (H,), cur)
    _check_gpu("h0", h0, torch.float32, (bsz, H, P, N), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, H, P), cur)
    if return_final_state and final_state is None:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=x.device)
    _check_gpu("final_state", final_state, torch.float32, (bsz, H, P, N), cur)
    d = ssd_desc(bsz, L, H, P, N, G, chunk, io)
    ws_bytes = lib.mssm_ssd_workspace_size(ctypes.byref(d))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    ws = (_ptr(workspace) if ws_bytes else None,
          workspace.numel() if (ws_bytes and workspace is not None) else 0, _stream_handle(stream))
    if trap:
        st = lib.mssm_ssd_trapezoidal_fwd(ctypes.byref(d), _ptr(x), _ptr(delta), _ptr(lam), _ptr(A), _ptr(B),
                                          _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(out), _ptr(final_state), *ws)
    else:
        st = lib.mssm_ssd_fwd(ctypes.byref(d), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                              _ptr(h0), _ptr(out), _ptr(final_state), *ws)
    if st != MSSM_OK:
        raise MssmError(st, fn)
    return (out, final_state) if return_final_state else out


def selective_state_update(state, x, delta, A, B, C, D=None, z=None, out=None, stream=None):
    """Advance a Mamba-1 state by seqlen tokens in place (mssm_selective_state_update).

    state: [batch, dim, dstate] float32 (overwritten); x, delta, z: [batch, seqlen, dim];
    B, C: [batch, seqlen, dstate] (float32 or bfloat16, all alike); A: [dim, dstate]; D: [dim].
    Returns out [batch, seqlen, dim].
    """
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [batch, seqlen, dim]")
    bsz, L, dm = x.shape
    if A.dim() != 2 or A.shape[0] != dm:
        raise ValueError("A must be [dim, dstate]")
    N = A.shape[1]
    io = _io_code(x.dtype)
    cur = _torch().cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, dm)), ("delta", delta, (bsz, L, dm)), ("z", z, (bsz, L, dm)),
                           ("B", B, (bsz, L, N)), ("C", C, (bsz, L, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    _check_gpu("state", state, torch.float32, (bsz, dm, N), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, dm), cur)
    d = scan_desc(bsz, L, dm, N, io)
    st = lib.mssm_selective_state_update(ctypes.byref(d), _ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B),
                                         _ptr(C), _ptr(D), _ptr(z), _ptr(out), _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_state_update")
    return out


def selective_state_update_conv(state, conv_state, xin, conv_w, conv_b, delta, A, B, C, D=None, z=None, out=None,
                                stream=None):
    """Token-by-token update with the short causal convolution in front (mssm_selective_state_update_conv).

    state [batch, dim, dstate] float32 and conv_state [batch, W-1, dim] (xin's dtype; None when W == 1) are
    advanced in place; xin, delta, z: [batch, T, dim]; conv_w [dim, W] float32; conv_b [dim] or None.
    Returns out [batch, T, dim]."""
    torch = _torch()
    if xin.dim() != 3:
        raise ValueError("xin must be [batch, tokens, dim]")
    bsz, T, dm = xin.shape
    N = A.shape[1]
    W = conv_w.shape[1]
    io = _io_code(xin.dtype)
    cur = _torch().cuda.current_device()
    for name, t, shape in (("xin", xin, (bsz, T, dm)), ("delta", delta, (bsz, T, dm)), ("z", z, (bsz, T, dm)),
                           ("B", B, (bsz, T, N)), ("C", C, (bsz, T, N)),
                           ("conv_state", conv_state, (bsz, W - 1, dm))):
        _check_gpu(name, t, xin.dtype, shape, cur)
    _check_gpu("state", state, torch.float32, (bsz, dm, N), cur)
    _check_gpu("conv_w", conv_w, torch.float32, (dm, W), cur)
    _check_gpu("conv_b", conv_b, torch.float32, (dm,), cur)
    _check_gpu("A", A, torch.float32, (dm, N), cur)
    _check_gpu("D", D, torch.float32, (dm,), cur)
    if out is None:
        out = torch.empty_like(xin)
    _check_gpu("out", out, xin.dtype, (bsz, T, dm), cur)
    d = scan_desc(bsz, T, dm, N, io)
    st = lib.mssm_selective_state_update_conv(ctypes.byref(d), W, _ptr(state), _ptr(conv_state), _ptr(xin),
                                              _ptr(conv_w), _ptr(conv_b), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                              _ptr(D), _ptr(z), _ptr(out), _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_selective_state_update_conv")
    return out


def ssd_state_update(state, x, delta, A, B, C, D=None, z=None, out=None, stream=None):
    """Advance a multi-head (scalar A) state by seqlen tokens in place (mssm_ssd_state_update).

    state: [batch, nheads, headdim, dstate] float32 (overwritten); x, z: [batch, seqlen, nheads, headdim];
    delta: [batch, seqlen, nheads]; B, C: [batch, seqlen, ngroups, dstate]; A, D: [nheads].
    Returns out [batch, seqlen, nheads, headdim].
    """
    return _ssd_update_call("mssm_ssd_state_update", state, None, None, x, delta, None, A, B, C, D, z, out, stream)


def ssd_trapezoidal_state_update(state, x, delta, lam, A, B, C, D=None, z=None, x_prev=None, B_prev=None,
                                 out=None, stream=None):
    """Advance a multi-head state by seqlen tokens in place under the Mamba-3 SISO rule
    (mssm_ssd_trapezoidal_state_update).

    As ``ssd_state_update`` plus lam [batch, seqlen, nheads] and the previous token's x_prev
    [batch, nheads, headdim] and B_prev [batch, ngroups, dstate] (None: no previous token).
    """
    return _ssd_update_call("mssm_ssd_trapezoidal_state_update", state, x_prev, B_prev, x, delta, lam, A, B, C, D,
                            z, out, stream)


def mamba3_siso_update(state, x, delta, lam, A, omega, B, C, D=None, z=None, x_prev=None, B_prev=None, out=None,
                       stream=None):
    """Advance a multi-head state by seqlen tokens in place under the Mamba-3 SISO recurrence with a
    complex-valued state (mssm_mamba3_siso_update): the exponential-trapezoidal rule, each state pair
    rotated by delta * omega per step.

    As ``ssd_trapezoidal_state_update`` plus omega [nheads, dstate / 2] float32; dstate must be even.
    With seqlen = L it is also the sequence form (state in: h0; state out: the final state).
    """
    return _ssd_update_call("mssm_mamba3_siso_update", state, x_prev, B_prev, x, delta, lam, A, B, C, D, z, out,
                            stream, omega=omega)


def _ssd_update_call(fn, state, x_prev, B_prev, x, delta, lam, A, B, C, D, z, out, stream, omega=None):
    torch = _torch()
    if x.dim() != 4:
        raise ValueError("x must be [batch, seqlen, nheads, headdim]")
    bsz, L, H, P = x.shape
    if B.dim() != 4:
        raise ValueError("B must be [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2], B.shape[3]
    io = _io_code(x.dtype)
    trap = fn in ("mssm_ssd_trapezoidal_state_update", "mssm_mamba3_siso_update")
    if trap and lam is None:
        raise ValueError("lam is required")
    if fn == "mssm_mamba3_siso_update" and omega is None:
        raise ValueError("omega is required")
    cur = _torch().cuda.current_device()
    for name, t, shape in (("x", x, (bsz, L, H, P)), ("z", z, (bsz, L, H, P)), ("delta", delta, (bsz, L, H)),
                           ("lam", lam, (bsz, L, H)), ("B", B, (bsz, L, G, N)), ("C", C, (bsz, L, G, N)),
                           ("x_prev", x_prev, (bsz, H, P)), ("B_prev", B_prev, (bsz, G, N))):
        _check_gpu(name, t, x.dtype, shape, cur)
    _check_gpu("A", A, torch.float32, (H,), cur)
    _check_gpu("D", D, torch.float32, (H,), cur)
    _check_gpu("state", state, torch.float32, (bsz, H, P, N), cur)
    _check_gpu("omega", omega, torch.float32, (H, N // 2), cur)
    if out is None:
        out = torch.empty_like(x)
    _check_gpu("out", out, x.dtype, (bsz, L, H, P), cur)
    d = ssd_desc(bsz, L, H, P, N, G, 0, io)
    if fn == "mssm_mamba3_siso_update":
        st = lib.mssm_mamba3_siso_update(ctypes.byref(d), _ptr(state), _ptr(x_prev), _ptr(B_prev), _ptr(x),
                                         _ptr(delta), _ptr(lam), _ptr(A), _ptr(omega), _ptr(B), _ptr(C), _ptr(D),
                                         _ptr(z), _ptr(out), _stream_handle(stream))
    elif trap:
        st = lib.mssm_ssd_trapezoidal_state_update(ctypes.byref(d), _ptr(state), _ptr(x_prev), _ptr(B_prev), _ptr(x),
                                                   _ptr(delta), _ptr(lam), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                                   _ptr(z), _ptr(out), _stream_handle(stream))
    else:
        st = lib.mssm_ssd_state_update(ctypes.byref(d), _ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B),
                                       _ptr(C), _ptr(D), _ptr(z), _ptr(out), _stream_handle(stream))
    if st != MSSM_OK:
        raise MssmError(st, fn)
    return out


# --------------------------------------------------------------------------
# Around the scan: embedding, norm, loss
# --------------------------------------------------------------------------
# (a decode step's call is dominated by what happens here on the host: one dictionary lookup instead of
# comparisons, no check twice, memory shaped after a tensor at hand where there is one)
_CODES = {}


def _codes(io_dtype) -> int:
    code = _CODES.get(io_dtype)
    if code is None:
        code = _CODES[io_dtype] = _io_code(io_dtype)
    return code


def _id_bytes(name, ids) -> int:
    torch = _torch()
    if ids.dtype is torch.int64:
        return 8
    if ids.dtype is torch.int32:
        return 4
    raise TypeError(f"{name} must be int32 or int64, got {ids.dtype}")


def _grad_code(name, t, io_dtype) -> int:
    if t.dtype != io_dtype and t.dtype != _torch().float32:
        raise TypeError(f"{name} must be {io_dtype} or torch.float32, got {t.dtype}")
    return _codes(t.dtype)


def _check_place(name, t, cur):
    """_check_gpu for a tensor whose own type and shape define the problem."""
    if t.get_device() != cur or not t.is_contiguous():
        _check_gpu(name, t, t.dtype, t.shape, cur)


def _stream_on(stream, cur) -> int:
    """_stream_handle with the current device known."""
    return _torch()._C._cuda_getCurrentRawStream(cur) if stream is None else _stream_handle(stream)


def _empty(stream, shape, dtype, like=None):
    """A new tensor on the current GPU (like: one of this shape and type), in the memory pool of the stream that
    the call runs on: memory of the current stream's pool could still be in use there, or be handed out again
    while the call runs."""
    torch = _torch()
    if stream is None:
        return torch.empty_like(like) if like is not None else torch.empty(shape, dtype=dtype, device="cuda")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace(need, workspace, stream):
    """(pointer, bytes, tensor to keep) of a call's workspace, allocated when none is given."""
    torch = _torch()
    if need == 0:
        return None, 0, None
    if workspace is None:
        workspace = _empty(stream, need, torch.uint8)
    elif workspace.get_device() != torch.cuda.current_device():
        raise ValueError("workspace must be on the current GPU")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def embedding_bwd_workspace_size(tokens, vocab, dim, io_dtype=MSSM_BF16) -> int:
    d = EmbeddingDesc(tokens, vocab, dim, 1.0, io_dtype, 8, 0)
    return lib.mssm_embedding_bwd_workspace_size(ctypes.byref(d))


def embedding_fwd(ids, weight, scale: float = 1.0, out=None, stream=None):
    """scale * weight[ids] (mssm_embedding_fwd).

    ids: int32 or int64 of any shape; weight: [vocab, dim] float32 or bfloat16.  An id outside
    [0, vocab) gives a row of zeros.  Returns out [*ids.shape, dim] in weight's type."""
    torch = _torch()
    if weight.dim() != 2:
        raise ValueError("weight must be [vocab, dim]")
    vocab, dim = weight.shape
    io, nb = _codes(weight.dtype), _id_bytes("ids", ids)
    cur = torch.cuda.current_device()
    _check_place("ids", ids, cur)
    _check_place("weight", weight, cur)
    shape = (*ids.shape, dim)
    if out is None:
        out = _empty(stream, shape, weight.dtype)
    else:
        _check_gpu("out", out, weight.dtype, shape, cur)
    d = EmbeddingDesc(ids.numel(), vocab, dim, scale, io, nb, 0)
    st = lib.mssm_embedding_fwd(ctypes.byref(d), ids.data_ptr(), weight.data_ptr(), out.data_ptr(),
                                _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_embedding_fwd")
    return out


def embedding_bwd(ids, dout, vocab: int, scale: float = 1.0, dweight=None, accumulate: bool = False, workspace=None,
                  stream=None):
    """Gradient of embedding_fwd's weight (mssm_embedding_bwd): row v is scale * the sum of dout over the
    tokens with id v, in the same order on every run.

    ids: int32 or int64; dout: [*ids.shape, dim].  dweight: [vocab, dim] in dout's type or float32 (allocated
    in dout's type when None), overwritten, or added to when accumulate.  Returns dweight."""
    torch = _torch()
    if dout.dim() != ids.dim() + 1:
        raise ValueError("dout must be [*ids.shape, dim]")
    dim = dout.shape[-1]
    io, nb = _codes(dout.dtype), _id_bytes("ids", ids)
    cur = torch.cuda.current_device()
    _check_place("ids", ids, cur)
    _check_gpu("dout", dout, dout.dtype, (*ids.shape, dim), cur)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate adds to dweight, which must be given")
        dweight = _empty(stream, (vocab, dim), dout.dtype)
    gd = _grad_code("dweight", dweight, dout.dtype)
    _check_gpu("dweight", dweight, dweight.dtype, (vocab, dim), cur)
    d = EmbeddingDesc(ids.numel(), vocab, dim, scale, io, nb, 0)
    ws, ws_bytes, _keep = _workspace(lib.mssm_embedding_bwd_workspace_size(ctypes.byref(d)), workspace, stream)
    st = lib.mssm_embedding_bwd(ctypes.byref(d), _ptr(ids), _ptr(dout), _ptr(dweight), gd, int(accumulate), ws,
                                ws_bytes, _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_embedding_bwd")
    return dweight


def norm_bwd_workspace_size(rows, dim) -> int:
    d = NormDesc(rows, dim, 1e-5, MSSM_LAYER_NORM, MSSM_F32, MSSM_F32, 0)
    return lib.mssm_norm_bwd_workspace_size(ctypes.byref(d))


def layer_norm_fwd(x, weight, bias=None, residual=None, eps: float = 1e-5, return_residual: bool = False,
                   residual_dtype=None, return_stats: bool = False, out=None, residual_out=None, stream=None):
    """Layer norm over the last axis of h = x + residual (mssm_norm_fwd).

    x: [..., dim] float32 or bfloat16; weight, bias: [dim] float32; residual: x's shape, x's type or float32.
    h is kept in residual_out (residual's type, else residual_dtype, else x's), and what is normalised is h as kept.
    Returns out, and after it residual_out with return_residual and (mean, rstd), float32 of x's leading
    shape, with return_stats: the gradients take them.  Without a residual h is x itself, unless
    return_residual."""
    return _norm_fwd(MSSM_LAYER_NORM, x, weight, bias, residual, eps, return_residual, residual_dtype, return_stats,
                     out, residual_out, stream)


def rms_norm_fwd(x, weight, residual=None, eps: float = 1e-5, return_residual: bool = False, residual_dtype=None,
                 return_stats: bool = False, out=None, residual_out=None, stream=None):
    """RMS norm over the last axis of h = x + residual (mssm_norm_fwd): as layer_norm_fwd without the mean and
    the bias.  Returns out, then residual_out with return_residual, then rstd with return_stats."""
    return _norm_fwd(MSSM_RMS_NORM, x, weight, None, residual, eps, return_residual, residual_dtype, return_stats,
                     out, residual_out, stream)


def _norm_fwd(kind, x, weight, bias, residual, eps, return_residual, residual_dtype, return_stats, out, residual_out,
              stream, fp8=False):
    torch = _torch()
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    shape, dim, xt = x.shape, x.shape[-1], x.dtype
    rows = x.numel() // dim if dim else 0
    io = _codes(xt)
    cur = torch.cuda.current_device()
    _check_place("x", x, cur)
    _check_gpu("weight", weight, torch.float32, (dim,), cur)
    if bias is not None:
        _check_gpu("bias", bias, torch.float32, (dim,), cur)
    rdt = residual.dtype if residual is not None else (residual_out.dtype if residual_out is not None else
                                                       (residual_dtype or xt))
    if residual_dtype is not None and residual_dtype != rdt:
        raise TypeError(f"residual_dtype is {residual_dtype}, but the residual is {rdt}")
    res = _res_code(rdt, xt)
    if residual is not None:
        _check_gpu("residual", residual, rdt, shape, cur)
    if fp8:
        if out is None:
            out = _fp8_empty(stream, rows, dim, False, x)
        else:
            _fp8_rows("out", out, dim, False, cur, rows)
    elif out is None:
        out = _empty(stream, shape, xt, x)
    else:
        _check_gpu("out", out, xt, shape, cur)
    if residual_out is not None:
        _check_gpu("residual_out", residual_out, rdt, shape, cur)
    elif residual is not None:
        residual_out = _empty(stream, shape, rdt, residual)
    elif return_residual:
        residual_out = _empty(stream, shape, rdt)
    mean = rstd = None
    if return_stats:
        rstd = _empty(stream, shape[:-1], torch.float32)
        if kind == MSSM_LAYER_NORM:
            mean = _empty(stream, shape[:-1], torch.float32, rstd)
    d = NormDesc(rows, dim, eps, kind, io, res, 0)
    if fp8:
        st = lib.mssm_norm_fp8_fwd(ctypes.byref(d), x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias),
                                   out.codes.data_ptr(), out.scales.data_ptr(), _ptr(residual_out), _ptr(mean),
                                   _ptr(rstd), _stream_on(stream, cur))
    else:
        st = lib.mssm_norm_fwd(ctypes.byref(d), x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias),
                               out.data_ptr(), _ptr(residual_out), _ptr(mean), _ptr(rstd), _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_norm_fp8_fwd" if fp8 else "mssm_norm_fwd")
    if return_stats:
        stats = (mean, rstd) if kind == MSSM_LAYER_NORM else (rstd,)
        return (out, residual_out, *stats) if return_residual else (out, *stats)
    return (out, residual_out) if return_residual else out


def _res_code(rdt, io_dtype) -> int:
    if rdt != io_dtype and rdt != _torch().float32:
        raise TypeError(f"the residual must be {io_dtype} or torch.float32, got {rdt}")
    return _codes(rdt)


def layer_norm_bwd(h, weight, mean, rstd, dout, dresidual=None, want_dresidual: bool = False, want_dbias: bool = True,
                   dx=None, workspace=None, stream=None):
    """Gradients of layer_norm_fwd (mssm_norm_bwd).

    h: what was normalised, residual_out of the forward (or x when there was none); mean, rstd: its
    statistics; dout: gradient of out; dresidual: gradient of residual_out (h's type) or None.
    Returns a dict: dx (dout's type; the gradient of x and, when the types agree, of the residual), dresidual
    (the same in h's type, when want_dresidual), dweight and dbias (float32)."""
    return _norm_bwd(MSSM_LAYER_NORM, h, weight, mean, rstd, dout, dresidual, want_dresidual, want_dbias, dx,
                     workspace, stream)


def rms_norm_bwd(h, weight, rstd, dout, dresidual=None, want_dresidual: bool = False, dx=None, workspace=None,
                 stream=None):
    """Gradients of rms_norm_fwd (mssm_norm_bwd): as layer_norm_bwd without mean and dbias."""
    return _norm_bwd(MSSM_RMS_NORM, h, weight, None, rstd, dout, dresidual, want_dresidual, False, dx, workspace,
                     stream)


def _norm_bwd(kind, h, weight, mean, rstd, dout, dresidual, want_dresidual, want_dbias, dx, workspace, stream):
    torch = _torch()
    if h.dim() < 1:
        raise ValueError("h must be [..., dim]")
    shape, dim = h.shape, h.shape[-1]
    rows = h.numel() // dim if dim else 0
    io = _codes(dout.dtype)
    res = _res_code(h.dtype, dout.dtype)
    cur = torch.cuda.current_device()
    _check_place("h", h, cur)
    _check_gpu("dout", dout, dout.dtype, shape, cur)
    _check_gpu("dresidual", dresidual, h.dtype, shape, cur)
    _check_gpu("weight", weight, torch.float32, (dim,), cur)
    if kind == MSSM_LAYER_NORM and mean is None:
        raise ValueError("mean is required")
    _check_gpu("mean", mean, torch.float32, shape[:-1], cur)
    _check_gpu("rstd", rstd, torch.float32, shape[:-1], cur)
    if dx is None:
        dx = _empty(stream, shape, dout.dtype, dout)
    else:
        _check_gpu("dx", dx, dout.dtype, shape, cur)
    dres = _empty(stream, shape, h.dtype, h) if want_dresidual else None
    dweight = _empty(stream, (dim,), torch.float32)
    dbias = _empty(stream, (dim,), torch.float32) if want_dbias else None
    d = NormDesc(rows, dim, 1.0, kind, io, res, 0)
    ws, ws_bytes, _keep = _workspace(lib.mssm_norm_bwd_workspace_size(ctypes.byref(d)), workspace, stream)
    st = lib.mssm_norm_bwd(ctypes.byref(d), _ptr(h), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dout),
                           _ptr(dresidual), _ptr(dx), _ptr(dres), _ptr(dweight), _ptr(dbias), ws, ws_bytes,
                           _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_norm_bwd")
    return {"dx": dx, "dresidual": dres, "dweight": dweight, "dbias": dbias}


def linear_cross_entropy_fwd_workspace_size(tokens, vocab, dim, io_dtype=MSSM_BF16) -> int:
    d = CrossEntropyDesc(tokens, vocab, dim, -100, io_dtype, 8, 0)
    return lib.mssm_linear_cross_entropy_fwd_workspace_size(ctypes.byref(d))


def linear_cross_entropy_bwd_workspace_size(tokens, vocab, dim, io_dtype=MSSM_BF16, fine: bool = False) -> int:
    d = CrossEntropyDesc(tokens, vocab, dim, -100, io_dtype, 8, MSSM_CROSS_ENTROPY_FINE_G if fine else 0)
    return lib.mssm_linear_cross_entropy_bwd_workspace_size(ctypes.byref(d))


def _xent_args(x, weight, targets, ignore_id, cur, fine=False):
    if x.dim() < 1 or weight.dim() != 2 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be [..., dim] and weight [vocab, dim]")
    vocab, dim = weight.shape
    io, nb = _codes(x.dtype), _id_bytes("targets", targets)
    _check_place("x", x, cur)
    _check_gpu("weight", weight, x.dtype, (vocab, dim), cur)
    _check_gpu("targets", targets, targets.dtype, x.shape[:-1], cur)
    return CrossEntropyDesc(targets.numel(), vocab, dim, ignore_id, io, nb, MSSM_CROSS_ENTROPY_FINE_G if fine else 0)


def linear_cross_entropy_fwd(x, weight, targets, ignore_id: int = -100, loss=None, lse=None, workspace=None,
                             stream=None):
    """Cross entropy of softmax(x @ weight.T) against targets, token by token, without keeping the logits
    (mssm_linear_cross_entropy_fwd).

    x: [..., dim] and weight: [vocab, dim], float32 or bfloat16 alike; targets: int32 or int64 of x's leading
    shape.  A token whose target is ignore_id or outside [0, vocab) is left out: loss and lse 0.
    Returns (loss, lse), float32 of targets' shape; lse is log sum exp of the token's logits."""
    torch = _torch()
    cur = torch.cuda.current_device()
    d = _xent_args(x, weight, targets, ignore_id, cur)
    shape = tuple(targets.shape)
    loss = _empty(stream, shape, torch.float32) if loss is None else loss
    lse = _empty(stream, shape, torch.float32) if lse is None else lse
    _check_gpu("loss", loss, torch.float32, shape, cur)
    _check_gpu("lse", lse, torch.float32, shape, cur)
    ws, ws_bytes, _keep = _workspace(lib.mssm_linear_cross_entropy_fwd_workspace_size(ctypes.byref(d)), workspace,
                                     stream)
    st = lib.mssm_linear_cross_entropy_fwd(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(targets), _ptr(loss),
                                           _ptr(lse), ws, ws_bytes, _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_linear_cross_entropy_fwd")
    return loss, lse


def linear_cross_entropy_bwd(x, weight, targets, lse, dloss, dlse=None, ignore_id: int = -100, want_dx: bool = True,
                             want_dweight: bool = True, dx=None, dweight=None, accumulate: bool = False,
                             workspace=None, stream=None, fine: bool = False):
    """Gradients of sum(loss * dloss) + sum(lse * dlse) with respect to x and weight
    (mssm_linear_cross_entropy_bwd).

    lse: as linear_cross_entropy_fwd returned it; dloss, dlse: float32 of targets' shape (dlse None: zero).
    dweight: [vocab, dim] in x's type or float32 (allocated in x's type when None), overwritten, or added to
    when accumulate (a head tied to the embedding, several batches).  fine: with bfloat16 the logits' gradient
    keeps 16 bits before its products with weight and x, as it does anyway for up to 256 tokens, instead of
    bfloat16's 8.  Returns a dict of dx and dweight (None for one that is not wanted)."""
    torch = _torch()
    cur = torch.cuda.current_device()
    d = _xent_args(x, weight, targets, ignore_id, cur, fine)
    shape = tuple(targets.shape)
    _check_gpu("lse", lse, torch.float32, shape, cur)
    _check_gpu("dloss", dloss, torch.float32, shape, cur)
    _check_gpu("dlse", dlse, torch.float32, shape, cur)
    if not want_dx and not want_dweight:
        raise ValueError("nothing to compute: want_dx and want_dweight are both False")
    if want_dx:
        dx = _empty(stream, tuple(x.shape), x.dtype) if dx is None else dx
        _check_gpu("dx", dx, x.dtype, tuple(x.shape), cur)
    else:
        dx = None
    gd = d.io_dtype
    if want_dweight:
        if dweight is None:
            if accumulate:
                raise ValueError("accumulate adds to dweight, which must be given")
            dweight = _empty(stream, tuple(weight.shape), weight.dtype)
        gd = _grad_code("dweight", dweight, x.dtype)
        _check_gpu("dweight", dweight, dweight.dtype, tuple(weight.shape), cur)
    else:
        dweight = None
    ws, ws_bytes, _keep = _workspace(lib.mssm_linear_cross_entropy_bwd_workspace_size(ctypes.byref(d)), workspace,
                                     stream)
    st = lib.mssm_linear_cross_entropy_bwd(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(targets), _ptr(lse),
                                           _ptr(dloss), _ptr(dlse), _ptr(dx), _ptr(dweight), gd, int(accumulate), ws,
                                           ws_bytes, _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_linear_cross_entropy_bwd")
    return {"dx": dx, "dweight": dweight}


# --------------------------------------------------------------------------
# The 8-bit linear layer
# --------------------------------------------------------------------------
class Fp8Matrix(NamedTuple):
    """A matrix [rows, cols] in 8 bits (include/mssm.h).

    codes: float8_e4m3fn [rows, 128 * blocks], blocks = ceil(cols / 128), zeros past cols; scales: float8_e8m0fnu,
    a power of two for each block of 128 columns of a row, [blocks, rows rounded up to 4], or with square for
    each 128 x 128, [blocks, ceil(rows / 128)].  The values are codes * scales."""
    codes: Any
    scales: Any
    cols: int
    square: bool = False


def _fp8_shapes(rows, cols, square):
    blocks = -(-cols // 128)
    return (rows, 128 * blocks), (blocks, -(-rows // 128) if square else -(-rows // 4) * 4)


def _matrix_empty(stream, shape, dtype, on):
    """_empty, faster by a quarter (1.25 us instead of 1.7 on the host) for a matrix beside a tensor on its GPU."""
    if stream is None and len(shape) == 2:
        return _torch().empty_strided(shape, (shape[1], 1), dtype=dtype, device=on.device)
    return _empty(stream, shape, dtype)


def _fp8_empty(stream, rows, cols, square, on) -> Fp8Matrix:
    torch = _torch()
    codes, scales = _fp8_shapes(rows, cols, square)
    return Fp8Matrix(_matrix_empty(stream, codes, torch.float8_e4m3fn, on),
                     _matrix_empty(stream, scales, torch.float8_e8m0fnu, on), cols, square)


def _fp8_rows(name, m, cols, square, cur, rows=None) -> int:
    """Rows of an Fp8Matrix on the current GPU, whose columns, kind and rows are as given (None: its own)."""
    torch = _torch()
    if type(m) is Fp8Matrix:
        codes, scales, own, kind = m
        shape = codes.shape
        # (a decode step's call is dominated by what happens here: all in one go, and what is wrong found out below)
        if (len(shape) == 2 and 0 < own and (cols is None or own == cols) and (square is None or kind is square)
                and (rows is None or rows == shape[0])):
            want, lines = _fp8_shapes(shape[0], own, kind)
            if (shape == want and scales.shape == lines and codes.dtype is torch.float8_e4m3fn
                    and scales.dtype is torch.float8_e8m0fnu and codes.get_device() == cur
                    and scales.get_device() == cur and codes.is_contiguous() and scales.is_contiguous()):
                return shape[0]
    if not isinstance(m, Fp8Matrix):
        raise TypeError(f"{name} must be an Fp8Matrix, got {type(m).__name__}")
    if m.codes.dim() != 2 or m.cols <= 0:
        raise ValueError(f"{name} must have codes [rows, 128 * blocks] and at least one column")
    if cols is not None and m.cols != cols:
        raise ValueError(f"{name} must have {cols} columns, got {m.cols}")
    if square is not None and bool(m.square) != square:
        raise ValueError(f"{name} must have a scale for each {'128 x 128' if square else '128 columns of a row'}")
    rows = m.codes.shape[0] if rows is None else rows
    want, lines = _fp8_shapes(rows, m.cols, bool(m.square))
    _check_gpu(name + ".codes", m.codes, torch.float8_e4m3fn, want, cur)
    _check_gpu(name + ".scales", m.scales, torch.float8_e8m0fnu, lines, cur)
    return rows


def _fp8_kind(square) -> int:
    return MSSM_FP8_SQUARE if square else MSSM_FP8_ROWS


def fp8_quantize(x, square: bool = False, transposed: bool = False, both: bool = False, out=None, stream=None):
    """x [rows, cols] (float32 or bfloat16) in 8 bits (mssm_fp8_quantize): an Fp8Matrix, with transposed that of
    x's transpose [cols, rows], with both the two of them from one read.

    square: a scale for each 128 x 128 (a weight, whose transpose then has the same values) instead of for
    each 128 columns of a row.  out: what is returned, to be written over."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    rows, cols = x.shape
    io = _codes(x.dtype)
    square = bool(square)
    cur = _torch().cuda.current_device()
    _check_place("x", x, cur)
    m = t = None
    if out is not None:
        m, t = out if both else (None, out) if transposed else (out, None)
    if both or not transposed:
        if m is None:
            m = _fp8_empty(stream, rows, cols, square, x)
        else:
            _fp8_rows("out", m, cols, square, cur, rows)
    if both or transposed:
        if rows == 0:
            raise ValueError("the transpose of no rows has no columns")
        if t is None:
            t = _fp8_empty(stream, cols, rows, square, x)
        else:
            _fp8_rows("out", t, rows, square, cur, cols)
    d = Fp8Desc(rows, cols, io, _fp8_kind(square), 0)
    st = lib.mssm_fp8_quantize(ctypes.byref(d), x.data_ptr(), _ptr(m and m.codes), _ptr(m and m.scales),
                               _ptr(t and t.codes), _ptr(t and t.scales), _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_fp8_quantize")
    return (m, t) if both else t if transposed else m


def fp8_transpose(m, out=None, stream=None) -> Fp8Matrix:
    """The transpose of an Fp8Matrix with scales of rows, with scales of its own rows (mssm_fp8_transpose): the
    values that m stands for, but below 2^-6 of their new block's scale, where they are rounded to 2^-9 of it."""
    cur = _torch().cuda.current_device()
    rows = _fp8_rows("m", m, None, False, cur)
    if rows == 0:
        raise ValueError("the transpose of no rows has no columns")
    if out is None:
        out = _fp8_empty(stream, m.cols, rows, False, m.codes)
    else:
        _fp8_rows("out", out, rows, False, cur, m.cols)
    d = Fp8Desc(rows, m.cols, MSSM_F32, MSSM_FP8_ROWS, 0)
    st = lib.mssm_fp8_transpose(ctypes.byref(d), m.codes.data_ptr(), m.scales.data_ptr(), out.codes.data_ptr(),
                                out.scales.data_ptr(), _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_fp8_transpose")
    return out


def fp8_dequantize(m, dtype=None, out=None, stream=None):
    """The values [rows, cols] that an Fp8Matrix stands for, in dtype (float32 or bfloat16, the default)
    (mssm_fp8_dequantize)."""
    torch = _torch()
    cur = torch.cuda.current_device()
    rows = _fp8_rows("m", m, None, None, cur)
    dtype = dtype or (torch.bfloat16 if out is None else out.dtype)
    io = _codes(dtype)
    if out is None:
        out = _matrix_empty(stream, (rows, m.cols), dtype, m.codes)
    else:
        _check_gpu("out", out, dtype, (rows, m.cols), cur)
    d = Fp8Desc(rows, m.cols, io, _fp8_kind(m.square), 0)
    st = lib.mssm_fp8_dequantize(ctypes.byref(d), m.codes.data_ptr(), m.scales.data_ptr(), out.data_ptr(),
                                 _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_fp8_dequantize")
    return out


def layer_norm_fp8_fwd(x, weight, bias=None, residual=None, eps: float = 1e-5, return_residual: bool = False,
                       residual_dtype=None, return_stats: bool = False, out=None, residual_out=None, stream=None):
    """layer_norm_fwd with its output in 8 bits, rounded once from float32 (mssm_norm_fp8_fwd): out is an Fp8Matrix
    [rows, dim], rows the product of x's leading sizes."""
    return _norm_fwd(MSSM_LAYER_NORM, x, weight, bias, residual, eps, return_residual, residual_dtype, return_stats,
                     out, residual_out, stream, fp8=True)


def rms_norm_fp8_fwd(x, weight, residual=None, eps: float = 1e-5, return_residual: bool = False, residual_dtype=None,
                     return_stats: bool = False, out=None, residual_out=None, stream=None):
    """rms_norm_fwd with its output in 8 bits, rounded once from float32 (mssm_norm_fp8_fwd): out is an Fp8Matrix
    [rows, dim], rows the product of x's leading sizes."""
    return _norm_fwd(MSSM_RMS_NORM, x, weight, None, residual, eps, return_residual, residual_dtype, return_stats,
                     out, residual_out, stream, fp8=True)


def fp8_linear_fwd_workspace_size(tokens, in_features, out_features, x_dtype=MSSM_E4M3, io_dtype=MSSM_BF16) -> int:
    d = Fp8LinearDesc(tokens, in_features, out_features, x_dtype, io_dtype, MSSM_FP8_SQUARE, 0)
    return lib.mssm_fp8_linear_fwd_workspace_size(ctypes.byref(d))


def fp8_linear_bwd_workspace_size(tokens, in_features, out_features, io_dtype=MSSM_BF16, grad_dtype=None,
                                  want_dx: bool = True, want_dweight: bool = True) -> int:
    d = Fp8LinearDesc(tokens, in_features, out_features, MSSM_E4M3, io_dtype, MSSM_FP8_SQUARE, 0)
    return lib.mssm_fp8_linear_bwd_workspace_size(ctypes.byref(d), int(want_dx), int(want_dweight),
                                                  io_dtype if grad_dtype is None else grad_dtype)


def fp8_linear_fwd(x, weight, out_dtype=None, out=None, workspace=None, stream=None):
    """x @ weight.T in 8 bits (mssm_fp8_linear_fwd).

    x: Fp8Matrix [tokens, in] with scales of rows, or a float32 or bfloat16 tensor [..., in], which is rounded
    as fp8_quantize would; weight: Fp8Matrix [out, in], square or not.  out_dtype: bfloat16 (the default)
    or float32, which also keeps more of the sums.  Returns [tokens, out], for a tensor x [..., out]."""
    torch = _torch()
    cur = torch.cuda.current_device()
    n = _fp8_rows("weight", weight, None, None, cur)
    k = weight.cols
    if isinstance(x, Fp8Matrix):
        tokens = _fp8_rows("x", x, k, False, cur)
        xd, xp, xs, shape = MSSM_E4M3, x.codes.data_ptr(), x.scales.data_ptr(), (tokens, n)
    else:
        if x.dim() < 1 or x.shape[-1] != k:
            raise ValueError(f"x must be [..., {k}]")
        xd, tokens = _codes(x.dtype), x.numel() // k
        _check_place("x", x, cur)
        xp, xs, shape = x.data_ptr(), None, (*x.shape[:-1], n)
    out_dtype = out_dtype or (torch.bfloat16 if out is None else out.dtype)
    io = _codes(out_dtype)
    if out is None:
        out = _matrix_empty(stream, shape, out_dtype, weight.codes)
    else:
        _check_gpu("out", out, out_dtype, shape, cur)
    d = Fp8LinearDesc(tokens, k, n, xd, io, _fp8_kind(weight.square), 0)
    ws, ws_bytes, _keep = _workspace(lib.mssm_fp8_linear_fwd_workspace_size(ctypes.byref(d)), workspace, stream)
    st = lib.mssm_fp8_linear_fwd(ctypes.byref(d), xp, xs, weight.codes.data_ptr(), weight.scales.data_ptr(),
                                 out.data_ptr(), ws, ws_bytes, _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_fp8_linear_fwd")
    return out


def fp8_linear_bwd(x, weight_t, dout, want_dx: bool = True, want_dweight: bool = True, dx=None, dweight=None,
                   dweight_dtype=None, accumulate: bool = False, workspace=None, stream=None):
    """Gradients of fp8_linear_fwd (mssm_fp8_linear_bwd), from its input as it was kept in 8 bits.

    x: Fp8Matrix [tokens, in] with scales of rows (None without dweight); weight_t: the transposed weight, Fp8Matrix
    [in, out], square or not (None without dx); dout: [tokens, out] (or any leading sizes), float32 or bfloat16,
    which is rounded to 8 bits along the sums that it enters.  dweight: [out, in] in dout's type or float32
    (allocated in dweight_dtype, else dout's, when None), overwritten, or added to when accumulate.
    Returns a dict of dx [tokens, in] (or dout's leading sizes) in dout's type and dweight (None for one that is not
    wanted)."""
    torch = _torch()
    cur = torch.cuda.current_device()
    if not want_dx and not want_dweight:
        raise ValueError("nothing to compute: want_dx and want_dweight are both False")
    if dout.dim() < 1 or dout.shape[-1] == 0:
        raise ValueError("dout must be [..., out]")
    io, n = _codes(dout.dtype), dout.shape[-1]
    tokens = dout.numel() // n
    _check_place("dout", dout, cur)
    if want_dx and weight_t is None:
        raise ValueError("weight_t is required for dx")
    if want_dweight and x is None:
        raise ValueError("x is required for dweight")
    k = None if weight_t is None else _fp8_rows("weight_t", weight_t, n, None, cur)
    square = weight_t is not None and bool(weight_t.square)
    if x is not None:
        _fp8_rows("x", x, k, False, cur, tokens)
        k = x.cols
    if want_dx:
        if dx is None:
            dx = _matrix_empty(stream, (*dout.shape[:-1], k), dout.dtype, dout)
        else:
            _check_gpu("dx", dx, dout.dtype, (*dout.shape[:-1], k), cur)
    else:
        dx = None
    gd = io
    if want_dweight:
        if dweight is None:
            if accumulate:
                raise ValueError("accumulate adds to dweight, which must be given")
            dweight = _matrix_empty(stream, (n, k), dweight_dtype or dout.dtype, dout)
        elif dweight_dtype is not None and dweight.dtype != dweight_dtype:
            raise TypeError(f"dweight_dtype is {dweight_dtype}, but dweight is {dweight.dtype}")
        gd = _grad_code("dweight", dweight, dout.dtype)
        _check_gpu("dweight", dweight, dweight.dtype, (n, k), cur)
    else:
        dweight = None
    d = Fp8LinearDesc(tokens, k, n, MSSM_E4M3, io, _fp8_kind(square), 0)
    ws, ws_bytes, _keep = _workspace(
        lib.mssm_fp8_linear_bwd_workspace_size(ctypes.byref(d), int(want_dx), int(want_dweight), gd), workspace, stream)
    st = lib.mssm_fp8_linear_bwd(ctypes.byref(d), _ptr(x and x.codes), _ptr(x and x.scales),
                                 _ptr(weight_t and weight_t.codes), _ptr(weight_t and weight_t.scales),
                                 dout.data_ptr(), _ptr(dx), _ptr(dweight), gd, int(accumulate), ws, ws_bytes,
                                 _stream_on(stream, cur))
    if st != MSSM_OK:
        raise MssmError(st, "mssm_fp8_linear_bwd")
    return {"dx": dx, "dweight": dweight}
