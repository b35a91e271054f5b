"""ctypes binding of libttt (include/ttt.h): argument marshalling only.

Every step of the layer runs in the CUDA library; this module checks shapes and
dtypes, allocates outputs with PyTorch (device memory and streams are PyTorch's
job here) and passes raw pointers.  There is no fallback: if the library is
missing or a tensor is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional

import torch

from .rotary import pair_bytes

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libttt.so")

TTT_F32, TTT_BF16 = 0, 1
STATUS = {0: "TTT_OK", -1: "TTT_ERR_ARG", -2: "TTT_ERR_UNSUPPORTED", -3: "TTT_ERR_ALIGN",
          -4: "TTT_ERR_LAUNCH", -5: "TTT_ERR_TIMEOUT", -6: "TTT_ERR_SCRATCH",
          -7: "TTT_ERR_RANGE"}

# every symbol include/ttt.h declares
EXPORTS = ("ttt_linear_fwd", "ttt_linear_seqpar_workspace", "ttt_linear_fwd_seqpar",
           "ttt_linear_fwd_seqpar_noalloc", "ttt_dwconv_fwd", "ttt_eta_gate",
           "ttt_mlp_fwd", "ttt_rope", "ttt_block_norm_fwd", "ttt_block_norm_bwd_workspace",
           "ttt_block_norm_bwd", "ttt_recurrence_fwd", "ttt_recurrence_bwd",
           "ttt_rope_axes", "ttt_short_conv_fwd", "ttt_short_conv_bwd_workspace", "ttt_short_conv_bwd",
           "ttt_selective_scan_fwd_workspace", "ttt_selective_scan_fwd", "ttt_selective_scan_bwd_workspace",
           "ttt_selective_scan_bwd", "ttt_sync_status", "ttt_status_str", "ttt_launch_count",
           "ttt_debug_wait_limit")


class LinearDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
                ("d", ctypes.c_int), ("mini_batch", ctypes.c_int), ("causal", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("w0_batch_stride", ctypes.c_longlong),
                ("loss", ctypes.c_int), ("epochs", ctypes.c_int),
                ("ln_gamma", ctypes.c_void_p), ("ln_beta", ctypes.c_void_p), ("ln_eps", ctypes.c_float)]

LOSSES = {"mse": 0, "dot": 1}


class DwconvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("height", ctypes.c_int),
                ("width", ctypes.c_int), ("d", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("loss", ctypes.c_int), ("epochs", ctypes.c_int),
                ("w0_batch_stride", ctypes.c_longlong)]


class MlpDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
                ("d", ctypes.c_int), ("m", ctypes.c_int), ("mini_batch", ctypes.c_int),
                ("causal", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("params_per_batch", ctypes.c_int), ("activation", ctypes.c_int),
                ("ln_gamma", ctypes.c_void_p), ("ln_beta", ctypes.c_void_p), ("ln_eps", ctypes.c_float)]

ACTIVATIONS = {"silu": 0, "gelu": 1}


class GateDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("dm", ctypes.c_int)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int),
                ("d", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inverse", ctypes.c_int), ("io_dtype", ctypes.c_int), ("table_rows", ctypes.c_int),
                ("period", ctypes.c_int), ("pos0", ctypes.c_longlong),
                ("positions_batch_stride", ctypes.c_longlong), ("strides", ctypes.c_longlong * 18)]


class BlockNormDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int), ("heads", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("post", ctypes.c_int), ("pre", ctypes.c_int), ("act", ctypes.c_int),
                ("post_eps", ctypes.c_float), ("pre_eps", ctypes.c_float), ("alpha", ctypes.c_float),
                ("strides", ctypes.c_longlong * 11)]


class BlockNormVectors(ctypes.Structure):
    """ttt_block_norm_params and ttt_block_norm_grads."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")]

NORMS = {"none": 0, "rms": 1, "layer": 2}
GATES = {"none": 0, "sigmoid": 1, "silu": 2, "gelu": 3}


class RecurrenceDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("mode", ctypes.c_int), ("strides", ctypes.c_longlong * 6)]

RECURRENCE_MODES = {"decay": 0, "sigmoid": 1, "mix": 2}
RECURRENCE_CHUNK = 128


class RopeAxesDesc(ctypes.Structure):
    _fields_ = [*RopeDesc._fields_, ("axes", ctypes.c_int), ("grid", ctypes.c_int * 4),
                ("positions_axis_stride", ctypes.c_longlong)]

ROPE_MAX_AXES = 4


class ShortConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int), ("width", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("act", ctypes.c_int), ("strides", ctypes.c_longlong * 4)]

CONV_ACTS = {"none": 0, "silu": 1}


class ScanDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int), ("N", ctypes.c_int), ("G", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("softplus", ctypes.c_int), ("strides", ctypes.c_longlong * 14)]


class ScanVectors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("A", "D", "delta_bias")]

SCAN_CHUNK = 32


class TTTError(RuntimeError):
    def __init__(self, fn, rc):
        self.code = rc
        super().__init__(f"{fn} returned {STATUS.get(rc, rc)}: {status_str(rc)}")


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libttt.so is missing ({LIB_PATH}); run "
                               "`python -m test_sequence_layers_gb300.build` first")
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, f = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float
        L.ttt_linear_fwd.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, f, fp, vp, fp, vp]
        L.ttt_linear_fwd.restype = ctypes.c_int
        L.ttt_linear_seqpar_workspace.argtypes = [ctypes.POINTER(LinearDesc)]
        L.ttt_linear_seqpar_workspace.restype = ctypes.c_size_t
        L.ttt_linear_fwd_seqpar.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, f, fp, vp, fp,
                                            vp, ctypes.c_size_t, vp]
        L.ttt_linear_fwd_seqpar.restype = ctypes.c_int
        L.ttt_linear_fwd_seqpar_noalloc.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, f, fp, vp,
                                                    fp, vp]
        L.ttt_linear_fwd_seqpar_noalloc.restype = ctypes.c_int
        L.ttt_dwconv_fwd.argtypes = [ctypes.POINTER(DwconvDesc), vp, vp, vp, fp, f, fp, vp, fp, vp]
        L.ttt_dwconv_fwd.restype = ctypes.c_int
        L.ttt_mlp_fwd.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, f, fp, fp, fp, fp,
                                  vp, fp, fp, fp, fp, vp]
        L.ttt_mlp_fwd.restype = ctypes.c_int
        L.ttt_eta_gate.argtypes = [ctypes.POINTER(GateDesc), vp, vp, f, fp, vp]
        L.ttt_eta_gate.restype = ctypes.c_int
        L.ttt_rope.argtypes = [ctypes.POINTER(RopeDesc), vp, vp, vp, fp, vp, vp, vp, vp, vp]
        L.ttt_rope.restype = ctypes.c_int
        L.ttt_block_norm_fwd.argtypes = [ctypes.POINTER(BlockNormDesc), ctypes.POINTER(BlockNormVectors), vp, vp, vp,
                                         vp, vp, fp, vp]
        L.ttt_block_norm_fwd.restype = ctypes.c_int
        L.ttt_block_norm_bwd_workspace.argtypes = [ctypes.POINTER(BlockNormDesc)]
        L.ttt_block_norm_bwd_workspace.restype = ctypes.c_size_t
        L.ttt_block_norm_bwd.argtypes = [ctypes.POINTER(BlockNormDesc), ctypes.POINTER(BlockNormVectors), vp, vp, vp,
                                         vp, vp, fp, vp, vp, vp, ctypes.POINTER(BlockNormVectors), vp,
                                         ctypes.c_size_t, vp]
        L.ttt_block_norm_bwd.restype = ctypes.c_int
        L.ttt_recurrence_fwd.argtypes = [ctypes.POINTER(RecurrenceDesc), vp, vp, vp, fp, vp, fp, fp, vp]
        L.ttt_recurrence_fwd.restype = ctypes.c_int
        L.ttt_recurrence_bwd.argtypes = [ctypes.POINTER(RecurrenceDesc), vp, vp, vp, vp, fp, fp, vp, vp, fp, vp]
        L.ttt_recurrence_bwd.restype = ctypes.c_int
        sz, P = ctypes.c_size_t, ctypes.POINTER
        L.ttt_rope_axes.argtypes = [P(RopeAxesDesc), ctypes.c_char_p, vp, vp, vp, fp, vp, vp, vp, vp, vp]
        L.ttt_short_conv_fwd.argtypes = [P(ShortConvDesc), vp, fp, fp, vp, vp, vp, vp, vp]
        L.ttt_short_conv_bwd.argtypes = [P(ShortConvDesc), vp, vp, fp, fp, vp, vp, fp, vp, fp, fp, fp, vp, sz, vp]
        L.ttt_selective_scan_fwd.argtypes = [P(ScanDesc), P(ScanVectors), vp, vp, vp, vp, vp, vp, fp, vp, fp, fp, vp, sz, vp]
        L.ttt_selective_scan_bwd.argtypes = [P(ScanDesc), P(ScanVectors), vp, vp, vp, vp, vp, vp, vp, fp, fp, vp, vp, vp, vp,
                                             vp, P(ScanVectors), fp, vp, sz, vp]
        for fn in (L.ttt_rope_axes, L.ttt_short_conv_fwd, L.ttt_short_conv_bwd, L.ttt_selective_scan_fwd,
                   L.ttt_selective_scan_bwd):
            fn.restype = ctypes.c_int
        for fn, desc in ((L.ttt_short_conv_bwd_workspace, ShortConvDesc), (L.ttt_selective_scan_fwd_workspace, ScanDesc),
                         (L.ttt_selective_scan_bwd_workspace, ScanDesc)):
            fn.argtypes, fn.restype = [P(desc)], sz
        L.ttt_sync_status.argtypes = [vp]
        L.ttt_sync_status.restype = ctypes.c_int
        L.ttt_status_str.argtypes = [ctypes.c_int]
        L.ttt_status_str.restype = ctypes.c_char_p
        L.ttt_launch_count.argtypes = []
        L.ttt_launch_count.restype = ctypes.c_ulonglong
        L.ttt_debug_wait_limit.argtypes = [ctypes.c_ulonglong]
        L.ttt_debug_wait_limit.restype = None
        _lib = L
    return _lib


def status_str(rc: int) -> str:
    return lib().ttt_status_str(rc).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_tokens(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B,H,T,d] tensor")
    if not (q.shape == k.shape == v.shape and q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share shape and dtype")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q, k, v must be bfloat16 or float32")
    return TTT_BF16 if q.dtype == torch.bfloat16 else TTT_F32


def _f32(t, name):
    if t is None:
        return None
    if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    return t


def _check_call(dev, stream, tensors, shapes):
    """Every tensor of a call lives on `dev` (the library launches on the current
    device, which the call makes `dev`), the stream belongs to it, and every given
    tensor has its expected shape.  Raises ValueError before anything is queued."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device} but q on {dev}: one device per call")
    for name, (t, shape) in shapes.items():
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device} but the tensors on {dev}")


def _each_tensor(x, act):
    if isinstance(x, (tuple, list)):
        for t in x:
            _each_tensor(t, act)
    elif hasattr(x, "record_stream"):
        act(x)


def _on_stream(stream, like, fn, *args):
    """fn(*args) on `stream`, another than the current one of `like`'s device, and safe
    for PyTorch's allocator: what the call allocates belongs to `stream` (memory that the
    current stream may still be using is not handed out, and a workspace is not reused
    before the kernels are done with it), the inputs are not reused before then either
    when the caller drops them, nor the results before the current stream's work on them."""
    if like.is_cuda:
        if stream.device != like.device:
            raise ValueError(f"the stream is on {stream.device} but the tensors on {like.device}")
        current = torch.cuda.current_stream(like.device)
        with torch.cuda.stream(stream):
            out = fn(*args)
        _each_tensor(args, lambda t: t.record_stream(stream))
        _each_tensor(out, lambda t: t.record_stream(current))
        return out
    return fn(*args)  # refuses


def _out_like_q(z, q):
    if z is not None and (z.dtype != q.dtype or not z.is_contiguous()):
        raise ValueError("z must be a contiguous tensor of q's dtype")


def _w0_stride(W0, B, H, d):
    if W0.shape == (H, d, d):
        return 0
    if W0.shape == (B, H, d, d):
        return H * d * d
    raise ValueError("W0 must be [H,d,d] or [B,H,d,d]")


def _linear_prologue(q, k, v, W0, eta, z, W_out, stream, ln_gamma=None, ln_beta=None):
    """Checks of every TTT-Linear wrapper; returns (io dtype, W0 batch stride)."""
    io = _check_tokens(q, k, v)
    B, H, T, d = q.shape
    for t, n in ((W0, "W0"), (eta, "eta"), (W_out, "W_out"), (ln_gamma, "ln_gamma"), (ln_beta, "ln_beta")):
        _f32(t, n)
    _check_call(q.device, stream,
                {"W0": W0, "eta": eta, "z": z, "W_out": W_out, "ln_gamma": ln_gamma, "ln_beta": ln_beta},
                {"eta": (eta, (B, H, T)), "z": (z, (B, H, T, d)), "W_out": (W_out, (B, H, d, d)),
                 "ln_gamma": (ln_gamma, (H, d)), "ln_beta": (ln_beta, (H, d))})
    _out_like_q(z, q)
    return io, _w0_stride(W0, B, H, d)


def ttt_linear_fwd(q, k, v, W0, mini_batch, causal=True, eta=None, eta_scalar=1.0,
                   z=None, W_out=None, want_W=True, stream=None, loss="mse", epochs=1,
                   ln_gamma=None, ln_beta=None, ln_eps=1e-6):
    """TTT-Linear forward.  q,k,v: [B,H,T,d] bf16 or fp32 CUDA tensors; W0: fp32
    [H,d,d] (shared over the batch) or [B,H,d,d]; eta: fp32 [B,H,T] or None;
    loss "mse" or "dot"; epochs > 1: repeated full-batch steps (causal=False,
    mini_batch >= T); ln_gamma, ln_beta: fp32 [H,d] for the inner model
    x + LN(x W).  Returns (z, W_final or None)."""
    if stream is not None:
        return _on_stream(stream, q, ttt_linear_fwd, q, k, v, W0, mini_batch, causal, eta, eta_scalar, z, W_out, want_W,
                          None, loss, epochs, ln_gamma, ln_beta, ln_eps)
    io, w0s = _linear_prologue(q, k, v, W0, eta, z, W_out, stream, ln_gamma, ln_beta)
    B, H, T, d = q.shape
    with torch.cuda.device(q.device):
        if z is None:
            z = torch.empty_like(q)
        if W_out is None and want_W:
            W_out = torch.empty((B, H, d, d), device=q.device, dtype=torch.float32)
        desc = LinearDesc(B, H, T, d, int(mini_batch), 1 if causal else 0, io, w0s, LOSSES[loss],
                          int(epochs), _ptr(ln_gamma), _ptr(ln_beta), float(ln_eps))
        rc = lib().ttt_linear_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                                  float(eta_scalar), _ptr(W0), _ptr(z), _ptr(W_out), _stream(stream))
    if rc != 0:
        raise TTTError("ttt_linear_fwd", rc)
    return z, W_out


def ttt_linear_seqpar_workspace(B, H, T, d, mini_batch, causal=True, dtype=torch.bfloat16,
                                loss="mse") -> int:
    """Workspace bytes ttt_linear_fwd_seqpar needs on the current device (0: the
    problem is not split)."""
    io = TTT_BF16 if dtype == torch.bfloat16 else TTT_F32
    desc = LinearDesc(B, H, T, d, int(mini_batch), 1 if causal else 0, io, 0, LOSSES[loss], 1)
    return int(lib().ttt_linear_seqpar_workspace(ctypes.byref(desc)))


def ttt_linear_fwd_seqpar(q, k, v, W0, mini_batch, causal=True, eta=None, eta_scalar=1.0,
                          z=None, W_out=None, want_W=True, workspace=None, stream=None, loss="mse"):
    """Sequence-parallel TTT-Linear forward (same arguments as ttt_linear_fwd).
    workspace: a CUDA uint8 tensor of at least ttt_linear_seqpar_workspace(...) bytes,
    allocated here when None.  Returns (z, W_final or None)."""
    if stream is not None:
        return _on_stream(stream, q, ttt_linear_fwd_seqpar, q, k, v, W0, mini_batch, causal, eta, eta_scalar, z, W_out,
                          want_W, workspace, None, loss)
    io, w0s = _linear_prologue(q, k, v, W0, eta, z, W_out, stream)
    _check_call(q.device, None, {"workspace": workspace}, {})
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    B, H, T, d = q.shape
    with torch.cuda.device(q.device):
        if z is None:
            z = torch.empty_like(q)
        if W_out is None and want_W:
            W_out = torch.empty((B, H, d, d), device=q.device, dtype=torch.float32)
        desc = LinearDesc(B, H, T, d, int(mini_batch), 1 if causal else 0, io, w0s, LOSSES[loss], 1)
        need = int(lib().ttt_linear_seqpar_workspace(ctypes.byref(desc)))
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib().ttt_linear_fwd_seqpar(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                                         float(eta_scalar), _ptr(W0), _ptr(z), _ptr(W_out),
                                         _ptr(workspace), nbytes, _stream(stream))
    if rc != 0:
        raise TTTError("ttt_linear_fwd_seqpar", rc)
    return z, W_out


def ttt_linear_fwd_seqpar_noalloc(q, k, v, W0, z, W_out, mini_batch, causal=True, eta=None,
                                  eta_scalar=1.0, stream=None, loss="mse"):
    """The sequence-parallel forward on the library's fixed scratch (no workspace,
    no allocation inside the call): z and W_out are the caller's output tensors."""
    if z is None:
        raise ValueError("z must be given (this entry point allocates nothing)")
    io, w0s = _linear_prologue(q, k, v, W0, eta, z, W_out, stream)
    B, H, T, d = q.shape
    with torch.cuda.device(q.device):
        desc = LinearDesc(B, H, T, d, int(mini_batch), 1 if causal else 0, io, w0s, LOSSES[loss], 1)
        rc = lib().ttt_linear_fwd_seqpar_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                                                 float(eta_scalar), _ptr(W0), _ptr(z), _ptr(W_out),
                                                 _stream(stream))
    if rc != 0:
        raise TTTError("ttt_linear_fwd_seqpar_noalloc", rc)
    return z, W_out


def ttt_dwconv_fwd(q, k, v, W0, height, width, eta=None, eta_scalar=1.0, loss="mse", epochs=1,
                   z=None, W_out=None, want_W=True, stream=None):
    """Depthwise 3x3 convolution inner model, full-batch inner GD.  q,k,v: [B,H,N,d]
    with N = height*width tokens in row-major grid order; W0: fp32 taps [H,9,d] or
    [B,H,9,d].  Returns (z, W_final [B,H,9,d] or None)."""
    if stream is not None:
        return _on_stream(stream, q, ttt_dwconv_fwd, q, k, v, W0, height, width, eta, eta_scalar, loss, epochs, z, W_out,
                          want_W)
    io = _check_tokens(q, k, v)
    B, H, N, d = q.shape
    if N != height * width:
        raise ValueError("q has N tokens, the grid height*width")
    for t, n in ((W0, "W0"), (eta, "eta"), (W_out, "W_out")):
        _f32(t, n)
    _check_call(q.device, stream, {"W0": W0, "eta": eta, "z": z, "W_out": W_out},
                {"eta": (eta, (B, H, N)), "z": (z, (B, H, N, d)), "W_out": (W_out, (B, H, 9, d))})
    _out_like_q(z, q)
    if W0.shape == (H, 9, d):
        w0s = 0
    elif W0.shape == (B, H, 9, d):
        w0s = H * 9 * d
    else:
        raise ValueError("W0 must be [H,9,d] or [B,H,9,d]")
    with torch.cuda.device(q.device):
        if z is None:
            z = torch.empty_like(q)
        if W_out is None and want_W:
            W_out = torch.empty((B, H, 9, d), device=q.device, dtype=torch.float32)
        desc = DwconvDesc(B, H, height, width, d, io, LOSSES[loss], int(epochs), w0s)
        rc = lib().ttt_dwconv_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                                  float(eta_scalar), _ptr(W0), _ptr(z), _ptr(W_out), _stream(stream))
    if rc != 0:
        raise TTTError("ttt_dwconv_fwd", rc)
    return z, W_out


def ttt_mlp_fwd(q, k, v, W1, c1, W2, c2, mini_batch, causal=True, eta=None, eta_scalar=0.1,
                z=None, outs=None, want_W=True, stream=None, activation="silu", ln_gamma=None,
                ln_beta=None, ln_eps=1e-6):
    """TTT-MLP forward, f(x) = act(x W1 + c1) W2 + c2, activation "silu" or "gelu"; with
    ln_gamma, ln_beta (fp32 [H,d]): f(x) = x + LN(act(x W1 + c1) W2 + c2).
    Parameters fp32, per head ([H,...]) or per (batch, head) ([B,H,...]).  outs: the
    final-weight tensors (W1, c1, W2, c2), each [B,H,...] fp32 or None.  Returns
    (z, (W1,c1,W2,c2) final or None)."""
    if stream is not None:
        return _on_stream(stream, q, ttt_mlp_fwd, q, k, v, W1, c1, W2, c2, mini_batch, causal, eta, eta_scalar, z, outs,
                          want_W, None, activation, ln_gamma, ln_beta, ln_eps)
    io = _check_tokens(q, k, v)
    B, H, T, d = q.shape
    W1, c1, W2, c2 = (_f32(t, n) for t, n in ((W1, "W1"), (c1, "c1"), (W2, "W2"), (c2, "c2")))
    eta = _f32(eta, "eta")
    ln_gamma, ln_beta = _f32(ln_gamma, "ln_gamma"), _f32(ln_beta, "ln_beta")
    m = W1.shape[-1]
    per_batch = 1 if W1.dim() == 4 else 0
    lead = (B, H) if per_batch else (H,)
    if (W1.shape != lead + (d, m) or c1.shape != lead + (m,) or W2.shape != lead + (m, d)
            or c2.shape != lead + (d,)):
        raise ValueError("inner weights must be W1 [..,d,m], c1 [..,m], W2 [..,m,d], c2 [..,d]")
    if outs is not None:
        if len(outs) != 4:
            raise ValueError("outs must be (W1, c1, W2, c2) final-weight tensors")
        for t, n in zip(outs, ("W1_out", "c1_out", "W2_out", "c2_out")):
            _f32(t, n)
    o = outs if outs is not None else (None, None, None, None)
    shapes = {"eta": (eta, (B, H, T)), "z": (z, (B, H, T, d)), "ln_gamma": (ln_gamma, (H, d)),
              "ln_beta": (ln_beta, (H, d))}
    for t, n, sh in zip(o, ("W1_out", "c1_out", "W2_out", "c2_out"), ((d, m), (m,), (m, d), (d,))):
        shapes[n] = (t, (B, H) + sh)
    _check_call(q.device, stream, {"W1": W1, "c1": c1, "W2": W2, "c2": c2, "eta": eta, "z": z,
                                   "ln_gamma": ln_gamma, "ln_beta": ln_beta,
                                   **dict(zip(("W1_out", "c1_out", "W2_out", "c2_out"), o))}, shapes)
    _out_like_q(z, q)
    with torch.cuda.device(q.device):
        if z is None:
            z = torch.empty_like(q)
        if outs is None and want_W:
            dev = q.device
            outs = (torch.empty((B, H, d, m), device=dev), torch.empty((B, H, m), device=dev),
                    torch.empty((B, H, m, d), device=dev), torch.empty((B, H, d), device=dev))
        o = outs if outs is not None else (None, None, None, None)
        desc = MlpDesc(B, H, T, d, m, int(mini_batch), 1 if causal else 0, io, per_batch,
                       ACTIVATIONS[activation], None if ln_gamma is None else ln_gamma.data_ptr(),
                       None if ln_beta is None else ln_beta.data_ptr(), float(ln_eps))
        rc = lib().ttt_mlp_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                               float(eta_scalar), _ptr(W1), _ptr(c1), _ptr(W2), _ptr(c2), _ptr(z),
                               *(_ptr(t) for t in o), _stream(stream))
    if rc != 0:
        raise TTTError("ttt_mlp_fwd", rc)
    return z, outs


def ttt_eta_gate(x, theta, eta_base=1.0, eta=None, stream=None):
    """Input-dependent inner learning rate eta[b,h,t] = eta_base * sigmoid(theta[h] .
    x[b,t]).  x: bf16 [B,T,dm] (the layer's input tokens); theta: bf16 [H,dm] (one
    vector per head).  Returns eta, fp32 [B,H,T] (the layout the TTT entry points
    read)."""
    if stream is not None:
        return _on_stream(stream, x, ttt_eta_gate, x, theta, eta_base, eta)
    for name, t in (("x", x), ("theta", theta)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor (no CPU path)")
    if x.dim() != 3 or theta.dim() != 2 or theta.shape[1] != x.shape[2]:
        raise ValueError("x must be [B,T,dm] and theta [H,dm]")
    B, T, dm = x.shape
    H = theta.shape[0]
    eta = _f32(eta, "eta")
    _check_call(x.device, stream, {"theta": theta, "eta": eta}, {"eta": (eta, (B, H, T))})
    with torch.cuda.device(x.device):
        if eta is None:
            eta = torch.empty((B, H, T), device=x.device, dtype=torch.float32)
        desc = GateDesc(B, T, H, dm)
        rc = lib().ttt_eta_gate(ctypes.byref(desc), _ptr(x), _ptr(theta), float(eta_base), _ptr(eta),
                                _stream(stream))
    if rc != 0:
        raise TTTError("ttt_eta_gate", rc)
    return eta


# ------------------------------------------------------- the streaming operators
#
# A decoding step calls these on a few hundred KB, where the host's time is the whole
# cost: descriptors are packed bytes, the current stream and device are read without their
# Python wrappers, each check is one expression that only asks why when it fails, and
# devices are compared by their numbers.

_IO = {torch.bfloat16: TTT_BF16, torch.float32: TTT_F32}
_ROPE_DESC, _NORM_DESC, _NORM_PAR = struct.Struct("@11i20q"), struct.Struct("@8i3f11q"), struct.Struct("@5Q")
_RECUR_DESC = struct.Struct("@5i6q")
_AXES_DESC, _CONV_DESC, _SCAN_DESC, _THREE = (struct.Struct("@11i20q5iq"), struct.Struct("@6i4q"), struct.Struct("@7i14q"),
                                              struct.Struct("@3Q"))
_NO_STRIDE2, _NO_STRIDE3 = (0, 0), (0, 0, 0)
_empty, _F32, _I64 = torch.empty, torch.float32, torch.int64
# the functions behind torch.cuda.current_stream and current_device, where PyTorch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda di: torch.cuda.current_stream(di).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_fns: dict = {}


def _fn(name):
    """An entry point taking addresses and packed descriptors as they are."""
    f = _fns.get(name)
    if f is None:
        f = lib()[name]
        n = {"ttt_rope": 10, "ttt_block_norm_fwd": 9, "ttt_block_norm_bwd": 15, "ttt_recurrence_fwd": 9,
             "ttt_recurrence_bwd": 11, "ttt_rope_axes": 11, "ttt_short_conv_fwd": 9, "ttt_short_conv_bwd": 15,
             "ttt_selective_scan_fwd": 15, "ttt_selective_scan_bwd": 21}[name]
        f.argtypes = [ctypes.c_void_p] * n
        f.restype = ctypes.c_int
        _fns[name] = f
    return f


def _workspace_bytes(name, desc):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = lib()[name]
        f.argtypes, f.restype = [ctypes.c_void_p], ctypes.c_size_t
    return f(desc)


def _norm_workspace(desc):
    return _workspace_bytes("ttt_block_norm_bwd_workspace", desc)


def _scratch(name, workspace, need, dev, di):
    """The caller's workspace, or one of the need's size from PyTorch's pool; (address, bytes, keeper)."""
    if workspace is None:
        if need == 0:
            return 0, 0, None
        workspace = _empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != di or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {name}'s device")
    return workspace.data_ptr(), workspace.nbytes, workspace


def _tokens(name, t, dims, like=None):
    """Why a token tensor is refused: CUDA, bf16 or fp32, `dims` dimensions, the last one
    contiguous; `like`: shares its dtype and device."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if t.dtype not in _IO:
        raise ValueError(f"{name} must be bfloat16 or float32")
    if t.stride()[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must share the dtype and device of the first tensor")


def _rows(name, t, like, shape, dt, di):
    """Strides (all but the last) of a token tensor of this shape, dtype and device."""
    st = t.stride()
    if t.dtype is not dt or t.get_device() != di or t.shape != shape or st[-1] != 1:
        _tokens(name, t, len(shape), like)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return st[:-1]


def _like(name, t, shape, dtype, di):
    """A contiguous tensor of the given shape, dtype and device."""
    if t.dtype is not dtype or t.get_device() != di or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{di}")
    return t


def _call(name, di, *args):
    """Runs one library entry point on device di's current stream."""
    f = _fns.get(name) or _fn(name)
    if _current_device() == di:
        rc = f(*args, _raw_stream(di))
    else:
        with torch.cuda.device(di):
            rc = f(*args, _raw_stream(di))
    if rc != 0:
        raise TTTError(name, rc)


def ttt_rope(q, k, v, table, positions=None, pos0=0, period=0, interleaved=False, inverse=False, q_out=None,
             k_out=None, v_out=None, stream=None):
    """Rotary positions on q and k, with the change of head layout; v (if given) is
    copied to its new layout in the same launch.

    q: [B,H,T,d] bf16 or fp32 with any strides as long as a head's features are
    contiguous (a [B,T,3,H,d] projection passes permuted views); k, v: [B,Hk,T,d] or None.
    table: fp32 [rows, rot/2, 2] cos and sin (rotary.rope_table).  positions: int64 [B,T]
    or [T] on the device, or None for pos0 + t; period > 0 takes them modulo period.
    interleaved: pairs (2i, 2i+1) instead of (i, i + rot/2).  inverse=True rotates back:
    the gradients of q, k, v from those of the outputs.  Outputs are contiguous
    [B,H,T,d] unless q_out, k_out, v_out are given (views whose dimensions
    step over those inside them; an output may be its own input, and shares memory with
    nothing else).  Returns (q_out, k_out, v_out).  A position outside the table gives NaN
    and TTT_ERR_RANGE from ttt_sync_status."""
    if stream is not None:
        return _on_stream(stream, q, ttt_rope, q, k, v, table, positions, pos0, period, interleaved, inverse, q_out,
                          k_out, v_out)
    return _rope(q, k, v, table, positions, pos0, period, interleaved, inverse, q_out, k_out, v_out, None, None)


def ttt_rope_axes(q, k, v, table, pair_axis, positions=None, grid=None, pos0=0, interleaved=False, inverse=False,
                  q_out=None, k_out=None, v_out=None, stream=None):
    """ttt_rope with several axes: pair i of a head turns by the token's position on axis
    pair_axis[i] (time, height, width, ...), rows of the table (rotary.rope_axes and
    rotary.rope_axes_table make both).  pair_axis: rot/2 small integers (bytes or a
    sequence).  positions: int64 [axes,B,T] or [axes,T] on the device; or grid: the
    extents of a row-major token grid, the last axis moving fastest, whose element pos0 + t
    token t is.  The rest as ttt_rope."""
    if stream is not None:
        return _on_stream(stream, q, ttt_rope_axes, q, k, v, table, pair_axis, positions, grid, pos0, interleaved, inverse,
                          q_out, k_out, v_out)
    if (positions is None) == (grid is None):
        raise ValueError("give either positions or grid")
    return _rope(q, k, v, table, positions, pos0, 0, interleaved, inverse, q_out, k_out, v_out, pair_axis, grid)


def _rope(q, k, v, table, positions, pos0, period, interleaved, inverse, q_out, k_out, v_out, pair_axis, grid):
    """ttt_rope, or with pair_axis ttt_rope_axes."""
    dt, dev, di, sq = q.dtype, q.device, q.get_device(), q.stride()
    io = _IO.get(dt)
    if io is None or not q.is_cuda or len(sq) != 4 or sq[3] != 1:
        _tokens("q", q, 4)
    B, H, T, d = shape = q.shape
    hk, sk, sv = 0, _NO_STRIDE3, _NO_STRIDE3
    if k is not None:
        hk = k.shape[1]
        sk = _rows("k", k, q, shape if hk == H else (B, hk, T, d), dt, di)
    if v is not None:
        if k is None:
            hk = v.shape[1]
        sv = _rows("v", v, q, shape if hk == H else (B, hk, T, d), dt, di)
    tshape = table.shape
    if (table.dtype is not _F32 or table.get_device() != di or len(tshape) != 3 or tshape[2] != 2
            or not table.is_contiguous()):
        raise ValueError("table must be a contiguous float32 [rows, rot/2, 2] tensor on q's device")
    pbs = 0
    if positions is not None:
        if positions.dtype is not _I64 or positions.get_device() != di or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int64 tensor on q's device")
        if pair_axis is not None:
            axes = positions.shape[0] if positions.dim() else 0
            pas = T
            if positions.shape == (axes, B, T):
                pbs, pas = T, B * T
            elif positions.shape != (axes, T):
                raise ValueError("positions must be [axes,B,T] or [axes,T]")
        elif positions.shape == (B, T):
            pbs = T
        elif positions.shape != (T,):
            raise ValueError("positions must be [B,T] or [T]")
    Td = T * d
    if q_out is None:
        q_out, so = _empty(shape, dtype=dt, device=dev), (H * Td, Td, d)
    else:
        so = _rows("q_out", q_out, q, shape, dt, di)
    sko = svo = _NO_STRIDE3
    if k is None:
        if k_out is not None:
            raise ValueError("k_out given without its input")
    elif k_out is None:
        k_out, sko = _empty(k.shape, dtype=dt, device=dev), (hk * Td, Td, d)
    else:
        sko = _rows("k_out", k_out, q, k.shape, dt, di)
    if v is None:
        if v_out is not None:
            raise ValueError("v_out given without its input")
    elif v_out is None:
        v_out, svo = _empty(v.shape, dtype=dt, device=dev), (hk * Td, Td, d)
    else:
        svo = _rows("v_out", v_out, q, v.shape, dt, di)
    if pair_axis is not None:
        if not isinstance(pair_axis, bytes):
            pair_axis = pair_bytes(pair_axis)
        if len(pair_axis) != tshape[1]:
            raise ValueError("pair_axis must name an axis for each of the table's pairs")
        if positions is None:
            axes, pas = len(grid), 0
        if not 1 <= axes <= ROPE_MAX_AXES:
            raise ValueError(f"there must be 1 to {ROPE_MAX_AXES} axes")
        extents = (0,) * ROPE_MAX_AXES if grid is None else (*grid, *(1,) * (ROPE_MAX_AXES - axes))
        desc = _AXES_DESC.pack(B, T, H, hk, d, 2 * tshape[1], interleaved, inverse, io, tshape[0], 0, pos0, pbs, *sq[:3], *sk,
                               *sv, *so, *sko, *svo, axes, *extents, pas)
        _call("ttt_rope_axes", di, desc, pair_axis, q.data_ptr(), 0 if k is None else k.data_ptr(),
              0 if v is None else v.data_ptr(), table.data_ptr(), 0 if positions is None else positions.data_ptr(),
              q_out.data_ptr(), 0 if k is None else k_out.data_ptr(), 0 if v is None else v_out.data_ptr())
        return q_out, k_out, v_out
    desc = _ROPE_DESC.pack(B, T, H, hk, d, 2 * tshape[1], interleaved, inverse, io, tshape[0], period, pos0, pbs,
                           *sq[:3], *sk, *sv, *so, *sko, *svo)
    _call("ttt_rope", di, desc, q.data_ptr(), 0 if k is None else k.data_ptr(), 0 if v is None else v.data_ptr(),
          table.data_ptr(), 0 if positions is None else positions.data_ptr(), q_out.data_ptr(),
          0 if k is None else k_out.data_ptr(), 0 if v is None else v_out.data_ptr())
    return q_out, k_out, v_out


def _vec(name, t, vshape, di):
    """The address of a parameter vector."""
    if t.dtype is not _F32 or t.get_device() != di or t.shape != vshape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [{vshape[0]}] tensor on cuda:{di}")
    return t.data_ptr()


def _norm_prologue(y, x, gate, act, post, pre, post_eps, pre_eps, alpha, w1, b1, scale, w2, b2, dh=None, du=None):
    """Checks of both block-norm wrappers; returns (token shape, dtype, device and its
    number, descriptor, parameters)."""
    dt, di, sy = y.dtype, y.get_device(), y.stride()
    io = _IO.get(dt)
    if io is None or not y.is_cuda or len(sy) not in (3, 4) or sy[-1] != 1:
        _tokens("y", y, 4 if len(sy) == 4 else 3)
    if len(sy) == 4:
        B, heads, T, d = y.shape
        D, sy = heads * d, sy[:3]
    else:
        B, T, D = y.shape
        heads, sy = 1, (sy[0], 0, sy[1])
    if (gate is None) != (act == "none"):
        raise ValueError('a gate goes with an act other than "none"')
    shape, vec = (B, T, D), (D,)
    sx = _NO_STRIDE2 if x is None else _rows("x", x, y, shape, dt, di)
    sg = _NO_STRIDE2 if gate is None else _rows("gate", gate, y, shape, dt, di)
    sdh = _NO_STRIDE2 if dh is None else _rows("dh", dh, y, shape, dt, di)
    sdu = _NO_STRIDE2 if du is None else _rows("du", du, y, shape, dt, di)
    par = _NORM_PAR.pack(0 if w1 is None else _vec("post_weight", w1, vec, di),
                         0 if b1 is None else _vec("post_bias", b1, vec, di),
                         0 if scale is None else _vec("scale", scale, vec, di),
                         0 if w2 is None else _vec("pre_weight", w2, vec, di),
                         0 if b2 is None else _vec("pre_bias", b2, vec, di))
    desc = _NORM_DESC.pack(B, T, D, heads, io, NORMS[post], NORMS[pre], GATES[act], post_eps, pre_eps, alpha, *sy, *sx,
                           *sg, *sdh, *sdu)
    return shape, dt, y.device, di, desc, par


def ttt_block_norm_fwd(y, x=None, gate=None, act=None, post="none", post_weight=None, post_bias=None, scale=None,
                       alpha=1.0, pre="none", pre_weight=None, pre_bias=None, post_eps=1e-6, pre_eps=1e-6,
                       want_stats=False, h=None, u=None, stats=None, stream=None):
    """The norms before and after a block, its gate and its residual in one pass:
        h = alpha x + scale * act(gate) * N_post(y),   u = N_pre(h)
    y: [B,T,D] or the layer's head-major [B,H,T,d] (D = H d); x, gate: [B,T,D] or None;
    bf16 or fp32, strided as long as the features are contiguous.  act "none", "sigmoid",
    "silu" or "gelu" (default: "silu" with a gate); post, pre "none", "rms" or "layer".
    Weights, biases and scale: fp32 [D] or None.  want_stats (or stats) for the backward
    pass.  h may be x.  Returns (h, u or None, stats or None)."""
    if stream is not None:
        return _on_stream(stream, y, ttt_block_norm_fwd, y, x, gate, act, post, post_weight, post_bias, scale, alpha,
                          pre, pre_weight, pre_bias, post_eps, pre_eps, want_stats, h, u, stats)
    if act is None:
        act = "none" if gate is None else "silu"
    shape, dt, dev, di, desc, par = _norm_prologue(y, x, gate, act, post, pre, post_eps, pre_eps, alpha, post_weight,
                                                   post_bias, scale, pre_weight, pre_bias)
    if pre != "none":
        u = _empty(shape, dtype=dt, device=dev) if u is None else _like("u", u, shape, dt, di)
    elif u is not None:
        raise ValueError("u is written with a pre norm only")
    if stats is not None:
        _like("stats", stats, (shape[0], shape[1], 4), _F32, di)
    elif want_stats:
        stats = _empty((shape[0], shape[1], 4), dtype=_F32, device=dev)
    h = _empty(shape, dtype=dt, device=dev) if h is None else _like("h", h, shape, dt, di)
    _call("ttt_block_norm_fwd", di, desc, par, y.data_ptr(), 0 if x is None else x.data_ptr(),
          0 if gate is None else gate.data_ptr(), h.data_ptr(), 0 if u is None else u.data_ptr(),
          0 if stats is None else stats.data_ptr())
    return h, u, stats


class BlockNormGrads(NamedTuple):
    """Gradients of ttt_block_norm_fwd's inputs, None for an absent input."""
    y: torch.Tensor
    x: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    post_weight: Optional[torch.Tensor]
    post_bias: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    pre_weight: Optional[torch.Tensor]
    pre_bias: Optional[torch.Tensor]


def ttt_block_norm_bwd(dh, du, y, stats, x=None, gate=None, act=None, post="none", post_weight=None, post_bias=None,
                       scale=None, alpha=1.0, pre="none", pre_weight=None, pre_bias=None, post_eps=1e-6, pre_eps=1e-6,
                       workspace=None, stream=None):
    """Gradients of ttt_block_norm_fwd from dh (or None) and du (None without a pre norm),
    the forward's inputs and its stats.  Returns BlockNormGrads: y's in y's shape
    (contiguous), fp32 [D] for every parameter vector given.  workspace: a CUDA uint8
    tensor of ttt_block_norm_bwd_workspace(...) bytes, allocated here when None."""
    if stream is not None:
        return _on_stream(stream, y, ttt_block_norm_bwd, dh, du, y, stats, x, gate, act, post, post_weight, post_bias,
                          scale, alpha, pre, pre_weight, pre_bias, post_eps, pre_eps, workspace)
    if act is None:
        act = "none" if gate is None else "silu"
    shape, dt, dev, di, desc, par = _norm_prologue(y, x, gate, act, post, pre, post_eps, pre_eps, alpha, post_weight,
                                                   post_bias, scale, pre_weight, pre_bias, dh, du)
    B, T, D = shape
    _like("stats", stats, (B, T, 4), _F32, di)
    dy = _empty(y.shape, dtype=dt, device=dev)
    dx = None if x is None else _empty(shape, dtype=dt, device=dev)
    dg = None if gate is None else _empty(shape, dtype=dt, device=dev)
    gv = [None if t is None else _empty(D, dtype=_F32, device=dev)
          for t in (post_weight, post_bias, scale, pre_weight, pre_bias)]
    if workspace is None:
        workspace = _empty(_norm_workspace(desc), dtype=torch.uint8, device=dev)
    elif workspace.get_device() != di or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on y's device")
    _call("ttt_block_norm_bwd", di, desc, par, 0 if dh is None else dh.data_ptr(),
          0 if du is None else du.data_ptr(), y.data_ptr(), 0 if x is None else x.data_ptr(),
          0 if gate is None else gate.data_ptr(), stats.data_ptr(), dy.data_ptr(), 0 if dx is None else dx.data_ptr(),
          0 if dg is None else dg.data_ptr(), _NORM_PAR.pack(*[0 if t is None else t.data_ptr() for t in gv]),
          workspace.data_ptr(), workspace.nbytes)
    return BlockNormGrads(dy, dx, dg, *gv)


def ttt_block_norm_bwd_workspace(B, T, D) -> int:
    """Workspace bytes of ttt_block_norm_bwd for B x T tokens of D features."""
    return _norm_workspace(_NORM_DESC.pack(B, T, D, 1, TTT_BF16, 0, 0, 0, 1e-6, 1e-6, 1.0, *[0] * 11))


def _recurrence_prologue(x, f, mode, reset, dh=None):
    """Checks of both recurrence wrappers; returns (shape, dtype, device and its
    number, descriptor)."""
    dt, di, sx = x.dtype, x.get_device(), x.stride()
    io = _IO.get(dt)
    if io is None or not x.is_cuda or len(sx) != 3 or sx[2] != 1:
        _tokens("x", x, 3)
    B, T, C = shape = x.shape
    sf = _rows("f", f, x, shape, dt, di)
    sd = _NO_STRIDE2 if dh is None else _rows("dh", dh, x, shape, dt, di)
    if reset is not None:
        if (reset.dtype not in (torch.bool, torch.uint8) or reset.get_device() != di or reset.shape != (B, T)
                or not reset.is_contiguous()):
            raise ValueError("reset must be a contiguous bool or uint8 [B,T] tensor on x's device")
    return shape, dt, x.device, di, _RECUR_DESC.pack(B, T, C, io, RECURRENCE_MODES[mode], sx[0], sx[1], *sf, *sd)


def ttt_recurrence_fwd(x, f, h0=None, mode="mix", reset=None, h=None, h_last=None, want_states=False, states=None,
                       stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + c_t x_t of every channel.  x, f: [B,T,C]
    bf16 or fp32, strided as long as the channels are contiguous.  mode "decay": a = f
    (|f| <= 1, see include/ttt.h), c = 1; "sigmoid": a = sigmoid(f), c = 1; "mix": a = sigmoid(f), c = 1 - a.  reset:
    bool or uint8 [B,T], True where a packed sequence begins (h_{t-1} taken as zero).
    h0: fp32 [B,C] or None; h_last may be h0 (a decoder's states stepped in place).
    want_states (or states) for the backward pass.  Returns (h, h_last, states or None)."""
    if stream is not None:
        return _on_stream(stream, x, ttt_recurrence_fwd, x, f, h0, mode, reset, h, h_last, want_states, states)
    shape, dt, dev, di, desc = _recurrence_prologue(x, f, mode, reset)
    B, T, C = shape
    if h0 is not None:
        _like("h0", h0, (B, C), _F32, di)
    if states is not None:
        _like("states", states, (B, -(-T // RECURRENCE_CHUNK), C), _F32, di)
    elif want_states:
        states = _empty((B, -(-T // RECURRENCE_CHUNK), C), dtype=_F32, device=dev)
    h = _empty(shape, dtype=dt, device=dev) if h is None else _like("h", h, shape, dt, di)
    h_last = _empty((B, C), dtype=_F32, device=dev) if h_last is None else _like("h_last", h_last, (B, C), _F32, di)
    _call("ttt_recurrence_fwd", di, desc, x.data_ptr(), f.data_ptr(), 0 if reset is None else reset.data_ptr(),
          0 if h0 is None else h0.data_ptr(), h.data_ptr(), h_last.data_ptr(), 0 if states is None else states.data_ptr())
    return h, h_last, states


def ttt_recurrence_bwd(dh, x, f, states, mode="mix", reset=None, dh_last=None, dx=None, df=None, dh0=None, stream=None):
    """Gradients of ttt_recurrence_fwd from dh ([B,T,C] or None) and dh_last (fp32 [B,C]
    or None), with the forward's inputs and the states it stored.  Returns (dx, df, dh0)."""
    if stream is not None:
        return _on_stream(stream, x, ttt_recurrence_bwd, dh, x, f, states, mode, reset, dh_last, dx, df, dh0)
    shape, dt, dev, di, desc = _recurrence_prologue(x, f, mode, reset, dh)
    B, T, C = shape
    _like("states", states, (B, -(-T // RECURRENCE_CHUNK), C), _F32, di)
    if dh_last is not None:
        _like("dh_last", dh_last, (B, C), _F32, di)
    dx = _empty(shape, dtype=dt, device=dev) if dx is None else _like("dx", dx, shape, dt, di)
    df = _empty(shape, dtype=dt, device=dev) if df is None else _like("df", df, shape, dt, di)
    dh0 = _empty((B, C), dtype=_F32, device=dev) if dh0 is None else _like("dh0", dh0, (B, C), _F32, di)
    _call("ttt_recurrence_bwd", di, desc, 0 if dh is None else dh.data_ptr(), x.data_ptr(), f.data_ptr(),
          0 if reset is None else reset.data_ptr(), states.data_ptr(), 0 if dh_last is None else dh_last.data_ptr(),
          dx.data_ptr(), df.data_ptr(), dh0.data_ptr())
    return dx, df, dh0


def _reset(reset, shape, di):
    if (reset.dtype not in (torch.bool, torch.uint8) or reset.get_device() != di or reset.shape != shape[:2]
            or not reset.is_contiguous()):
        raise ValueError("reset must be a contiguous bool or uint8 [B,T] tensor on x's device")


def _conv_prologue(x, weight, bias, act, reset, state, dy=None):
    """Checks of both convolution wrappers; returns (shape, width, dtype, device and its
    number, state shape, descriptor)."""
    dt, di, sx = x.dtype, x.get_device(), x.stride()
    io = _IO.get(dt)
    if io is None or not x.is_cuda or len(sx) != 3 or sx[2] != 1:
        _tokens("x", x, 3)
        sx = (*sx[:2], 1)
    B, T, C = shape = x.shape
    wshape = weight.shape
    if len(wshape) != 2:
        raise ValueError("weight must be [C,K]")
    K = wshape[1]
    if wshape[0] != C or weight.dtype is not _F32 or weight.get_device() != di or not weight.is_contiguous():
        _like("weight", weight, (C, K), _F32, di)
    if bias is not None and (bias.dtype is not _F32 or bias.get_device() != di or bias.shape != (C,) or not bias.is_contiguous()):
        _like("bias", bias, (C,), _F32, di)
    sd = _NO_STRIDE2 if dy is None else _rows("dy", dy, x, shape, dt, di)
    if reset is not None:
        _reset(reset, shape, di)
    sshape = (B, K - 1, C)
    if state is not None and (state.dtype is not dt or state.get_device() != di or state.shape != sshape
                              or not state.is_contiguous()):
        _like("state", state, sshape, dt, di)
    return shape, K, dt, x.device, di, sshape, _CONV_DESC.pack(B, T, C, K, io, CONV_ACTS[act], sx[0], sx[1], *sd)


def ttt_short_conv_fwd(x, weight, bias=None, act="silu", reset=None, state=None, y=None, want_state=False, state_out=None,
                       stream=None):
    """Short causal convolution of every channel along the tokens: y_t = act(bias + sum_j
    weight[:, j] x_{t-K+1+j}).  x: [B,T,C] bf16 or fp32, strided as long as the channels are
    contiguous; weight: fp32 [C,K], K up to 4; bias: fp32 [C] or None; act "none" or "silu".
    reset: bool or uint8 [B,T], True where a packed sequence begins (its tokens see zeros
    before it).  state: [B,K-1,C] in x's dtype, the inputs before the first token, oldest
    first, or None (zeros).  want_state (or state_out, which may be state: a decoder's
    states stepped in place) for the last K-1 inputs.  Returns (y, state_out or None)."""
    if stream is not None:
        return _on_stream(stream, x, ttt_short_conv_fwd, x, weight, bias, act, reset, state, y, want_state, state_out)
    shape, _, dt, dev, di, sshape, desc = _conv_prologue(x, weight, bias, act, reset, state)
    y = _empty(shape, dtype=dt, device=dev) if y is None else _like("y", y, shape, dt, di)
    if state_out is not None:
        _like("state_out", state_out, sshape, dt, di)
    elif want_state:
        state_out = _empty(sshape, dtype=dt, device=dev)
    _call("ttt_short_conv_fwd", di, desc, x.data_ptr(), weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
          0 if reset is None else reset.data_ptr(), 0 if state is None else state.data_ptr(), y.data_ptr(),
          0 if state_out is None else state_out.data_ptr())
    return y, state_out


class ShortConvGrads(NamedTuple):
    """Gradients of ttt_short_conv_fwd's inputs, None for an absent input."""
    x: torch.Tensor
    weight: torch.Tensor
    bias: Optional[torch.Tensor]
    state: Optional[torch.Tensor]


def ttt_short_conv_bwd(dy, x, weight, bias=None, act="silu", reset=None, state=None, dstate_out=None, workspace=None,
                       stream=None):
    """Gradients of ttt_short_conv_fwd from dy [B,T,C] and dstate_out (of state_out, fp32
    [B,K-1,C], or None), with the forward's inputs.  Returns ShortConvGrads: x's in x's
    dtype, the rest fp32.  workspace: a CUDA tensor of ttt_short_conv_bwd_workspace's bytes,
    allocated here when None."""
    if stream is not None:
        return _on_stream(stream, x, ttt_short_conv_bwd, dy, x, weight, bias, act, reset, state, dstate_out, workspace)
    shape, K, dt, dev, di, sshape, desc = _conv_prologue(x, weight, bias, act, reset, state, dy)
    if dstate_out is not None:
        _like("dstate_out", dstate_out, sshape, _F32, di)
    dx = _empty(shape, dtype=dt, device=dev)
    dw = _empty((shape[2], K), dtype=_F32, device=dev)
    db = None if bias is None else _empty(shape[2], dtype=_F32, device=dev)
    ds = None if state is None else _empty(sshape, dtype=_F32, device=dev)
    ws, nws, _keep = _scratch("x", workspace, _workspace_bytes("ttt_short_conv_bwd_workspace", desc), dev, di)
    _call("ttt_short_conv_bwd", di, desc, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
          0 if reset is None else reset.data_ptr(), 0 if state is None else state.data_ptr(),
          0 if dstate_out is None else dstate_out.data_ptr(), dx.data_ptr(), dw.data_ptr(), 0 if db is None else db.data_ptr(),
          0 if ds is None else ds.data_ptr(), ws, nws)
    return ShortConvGrads(dx, dw, db, ds)


def ttt_short_conv_bwd_workspace(B, T, C, K) -> int:
    """Workspace bytes of ttt_short_conv_bwd for B x T tokens of C channels, K taps."""
    return _workspace_bytes("ttt_short_conv_bwd_workspace", _CONV_DESC.pack(B, T, C, K, TTT_BF16, 0, 0, 0, 0, 0))


def _scan_prologue(x, delta, A, B, C, D, z, delta_bias, softplus, reset, dy=None):
    """Checks of both scan wrappers; returns (token shape, states' [C,N], B's and C's shapes,
    dtype, device and its number, descriptor, parameters)."""
    dt, di, sx = x.dtype, x.get_device(), x.stride()
    io = _IO.get(dt)
    if io is None or not x.is_cuda or len(sx) != 3 or sx[2] != 1:
        _tokens("x", x, 3)
        sx = (*sx[:2], 1)
    nb, T, ch = shape = x.shape
    cn, bshape = A.shape, B.shape
    if len(cn) != 2:
        raise ValueError("A must be [C,N]")
    N = cn[1]
    if cn[0] != ch or A.dtype is not _F32 or A.get_device() != di or not A.is_contiguous():
        _like("A", A, (ch, N), _F32, di)
    sdl = _rows("delta", delta, x, shape, dt, di)
    if len(bshape) == 4:
        G = bshape[2]
        bshape = (nb, T, G, N)
        sb, sc = _rows("B", B, x, bshape, dt, di), _rows("C", C, x, bshape, dt, di)
    else:
        G, bshape = 1, (nb, T, N)
        sb, sc = (*_rows("B", B, x, bshape, dt, di), 0), (*_rows("C", C, x, bshape, dt, di), 0)
    if G < 1 or ch % G:
        raise ValueError("the groups of B and C must divide the channels")
    sz = _NO_STRIDE2 if z is None else _rows("z", z, x, shape, dt, di)
    sdy = _NO_STRIDE2 if dy is None else _rows("dy", dy, x, shape, dt, di)
    if reset is not None:
        _reset(reset, shape, di)
    vec = (ch,)
    par = _THREE.pack(A.data_ptr(), 0 if D is None else _vec("D", D, vec, di),
                      0 if delta_bias is None else _vec("delta_bias", delta_bias, vec, di))
    desc = _SCAN_DESC.pack(nb, T, ch, N, G, io, bool(softplus), sx[0], sx[1], *sdl, *sz, *sdy, *sb, *sc)
    return shape, cn, bshape, dt, x.device, di, desc, par


def ttt_selective_scan_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, reset=None, h0=None, y=None,
                           h_last=None, want_states=False, states=None, workspace=None, stream=None):
    """Selective state space scan, N states a channel: with d = softplus(delta + delta_bias)
    (softplus=False: without it),
        h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t).
    x, delta, z: [B,T,C] bf16 or fp32, B, C: [B,T,N] or, for G groups of channels,
    [B,T,G,N], all strided as long as the last dimension is contiguous (slices of a
    projection); A: fp32 [C,N], D, delta_bias: fp32 [C] or None; z None: no gate.
    reset: bool or uint8 [B,T], True where a packed sequence begins.  h0: fp32 [B,C,N] or
    None; h_last may be h0 (a decoder's states stepped in place).  want_states (or states)
    for the backward pass.  Returns (y, h_last, states or None)."""
    if stream is not None:
        return _on_stream(stream, x, ttt_selective_scan_fwd, x, delta, A, B, C, D, z, delta_bias, softplus, reset, h0, y,
                          h_last, want_states, states, workspace)
    shape, cn, _, dt, dev, di, desc, par = _scan_prologue(x, delta, A, B, C, D, z, delta_bias, softplus, reset)
    nb, T, _ = shape
    hshape = (nb, *cn)
    if h0 is not None and (h0.dtype is not _F32 or h0.get_device() != di or h0.shape != hshape or not h0.is_contiguous()):
        _like("h0", h0, hshape, _F32, di)
    if states is not None:
        _like("states", states, (nb, -(-T // SCAN_CHUNK), *cn), _F32, di)
    elif want_states:
        states = _empty((nb, -(-T // SCAN_CHUNK), *cn), dtype=_F32, device=dev)
    y = _empty(shape, dtype=dt, device=dev) if y is None else _like("y", y, shape, dt, di)
    h_last = _empty(hshape, dtype=_F32, device=dev) if h_last is None else _like("h_last", h_last, hshape, _F32, di)
    ws = nws = 0
    if T > 1 or workspace is not None:  # a single token needs no workspace
        need = _workspace_bytes("ttt_selective_scan_fwd_workspace", desc) if workspace is None else 0
        ws, nws, _keep = _scratch("x", workspace, need, dev, di)
    _call("ttt_selective_scan_fwd", di, desc, par, x.data_ptr(), delta.data_ptr(), B.data_ptr(), C.data_ptr(),
          0 if z is None else z.data_ptr(), 0 if reset is None else reset.data_ptr(), 0 if h0 is None else h0.data_ptr(),
          y.data_ptr(), h_last.data_ptr(), 0 if states is None else states.data_ptr(), ws, nws)
    return y, h_last, states


class SelectiveScanGrads(NamedTuple):
    """Gradients of ttt_selective_scan_fwd's inputs, None for an absent input."""
    x: torch.Tensor
    delta: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    C: torch.Tensor
    D: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    delta_bias: Optional[torch.Tensor]
    h0: torch.Tensor


def ttt_selective_scan_bwd(dy, x, delta, A, B, C, states, D=None, z=None, delta_bias=None, softplus=True, reset=None,
                           dh_last=None, workspace=None, stream=None):
    """Gradients of ttt_selective_scan_fwd from dy [B,T,C] and dh_last (of h_last, fp32
    [B,C,N], or None), with the forward's inputs and the states it stored.  Returns
    SelectiveScanGrads: the token tensors' in their dtype, contiguous, the rest fp32 (h0's
    whether or not one was given).  workspace: a CUDA tensor of
    ttt_selective_scan_bwd_workspace's bytes, allocated here when None."""
    if stream is not None:
        return _on_stream(stream, x, ttt_selective_scan_bwd, dy, x, delta, A, B, C, states, D, z, delta_bias, softplus,
                          reset, dh_last, workspace)
    shape, cn, bshape, dt, dev, di, desc, par = _scan_prologue(x, delta, A, B, C, D, z, delta_bias, softplus, reset, dy)
    nb, T, ch = shape
    _like("states", states, (nb, -(-T // SCAN_CHUNK), *cn), _F32, di)
    if dh_last is not None:
        _like("dh_last", dh_last, (nb, *cn), _F32, di)
    dx, dd = _empty(shape, dtype=dt, device=dev), _empty(shape, dtype=dt, device=dev)
    dz = None if z is None else _empty(shape, dtype=dt, device=dev)
    dB, dC = _empty(bshape, dtype=dt, device=dev), _empty(bshape, dtype=dt, device=dev)
    dA, dh0 = _empty(cn, dtype=_F32, device=dev), _empty((nb, *cn), dtype=_F32, device=dev)
    dD = None if D is None else _empty(ch, dtype=_F32, device=dev)
    db = None if delta_bias is None else _empty(ch, dtype=_F32, device=dev)
    need = _workspace_bytes("ttt_selective_scan_bwd_workspace", desc) if workspace is None else 0
    ws, nws, _keep = _scratch("x", workspace, need, dev, di)
    grads = _THREE.pack(dA.data_ptr(), 0 if dD is None else dD.data_ptr(), 0 if db is None else db.data_ptr())
    _call("ttt_selective_scan_bwd", di, desc, par, dy.data_ptr(), x.data_ptr(), delta.data_ptr(), B.data_ptr(), C.data_ptr(),
          0 if z is None else z.data_ptr(), 0 if reset is None else reset.data_ptr(), states.data_ptr(),
          0 if dh_last is None else dh_last.data_ptr(), dx.data_ptr(), dd.data_ptr(), dB.data_ptr(), dC.data_ptr(),
          0 if dz is None else dz.data_ptr(), grads, dh0.data_ptr(), ws, nws)
    return SelectiveScanGrads(dx, dd, dA, dB, dC, dD, dz, db, dh0)


def ttt_selective_scan_fwd_workspace(B, T, C, N, G=1) -> int:
    """Workspace bytes of ttt_selective_scan_fwd."""
    return _workspace_bytes("ttt_selective_scan_fwd_workspace", _SCAN_DESC.pack(B, T, C, N, G, TTT_BF16, 1, *[0] * 14))


def ttt_selective_scan_bwd_workspace(B, T, C, N, G=1) -> int:
    """Workspace bytes of ttt_selective_scan_bwd."""
    return _workspace_bytes("ttt_selective_scan_bwd_workspace", _SCAN_DESC.pack(B, T, C, N, G, TTT_BF16, 1, *[0] * 14))


def ttt_sync_status(stream=None):
    """Waits for the stream; raises TTTError if a kernel wait timed out (code -5) or, reported
    after that, ttt_rope met a position outside its table (-7)."""
    rc = lib().ttt_sync_status(_stream(stream))
    if rc != 0:
        raise TTTError("ttt_sync_status", rc)


def ttt_launch_count() -> int:
    return int(lib().ttt_launch_count())


def ttt_debug_wait_limit(ns: int) -> None:
    """Test hook of the timeout path: ns > 0 makes the first consumer wait of the
    b = 16 and full-batch TTT-Linear kernels, of the full-batch TTT-MLP kernel and of the
    recurrence run out after ns nanoseconds (see include/ttt.h); 0 restores normal operation."""
    lib().ttt_debug_wait_limit(int(ns))
