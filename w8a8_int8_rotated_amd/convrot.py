"""Python binding of libconvrot (the C ABI in include/convrot.h).

Argument marshalling only: PyTorch provides device memory and the current HIP
stream; every step of the forward path runs in the library's HIP kernels.
The functions carry the C names.  If the library has not been built the first
call raises -- there is no fallback implementation.  They build no autograd graph,
whatever their inputs require: where an entry has a backward pass here
(convrot_rope_forward with inverse=True, convrot_qk_norm_rope_backward), a caller
joins the two in a torch.autograd.Function of their own.

stream=: the whole call, its copies and allocations among it, runs on that stream,
which must be ordered after whatever made the arguments.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libconvrot.so")

OK, EINVAL, EALIGN, EWORKSPACE, ELAYOUT, EUNSUPPORTED, EHIP = 0, -1, -2, -3, -4, -5, -6
F32, BF16, I8, I32, F8E4M3 = 0, 1, 2, 3, 4
OUT_MAJOR, IN_MAJOR = 0, 1
WEIGHTS_MAGIC = 0x38545243
WEIGHTS_VERSION = 2
ROT_REGULAR = 0x100          # rotation kind: regular H_4 Kronecker blocks
ROTATIONS = {"sylvester": 0, "regular": ROT_REGULAR}
FLAG_GELU = 1
FLAG_SWIGLU = 2
SWIGLU_PAIRS = 0x200         # weight flag: interleaved SwiGLU gate/up rows
FP8_MAGIC, FP8_VERSION = 0x38465243, 1
FP8_SCALES = {"f32": 0, "pow2": 1}
ROPE_MAGIC, ROPE_VERSION = 0x504F5243, 1
ROPE_PAIRINGS = {"interleaved": 0, "half": 1}
ROPE_SPECTRA = {"axis": 0, "whole": 1}
ROPE_MAX_AXES = 4
ROPE_INVERSE = 1
MOE_MAGIC, MOE_VERSION = 0x454F4D43, 1
MOE_SCORES = {"softmax": 0, "sigmoid": 1}
MOE_RENORMALIZE = 1
MOE_PASS = 64                # tokens of one pass over the experts; the workspace holds one

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_p = ctypes.c_void_p
_c_sz = ctypes.c_size_t


class convrot_weights(ctypes.Structure):
    _fields_ = [
        ("magic", ctypes.c_uint32),
        ("version", ctypes.c_uint32),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("block", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
    ]


_W = ctypes.POINTER(convrot_weights)


class convrot_fp8_weights(ctypes.Structure):
    _fields_ = [
        ("magic", ctypes.c_uint32),
        ("version", ctypes.c_uint32),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("scales", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
    ]


class convrot_rope(ctypes.Structure):
    _fields_ = [
        ("magic", ctypes.c_uint32),
        ("version", ctypes.c_uint32),
        ("axes", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("pairing", ctypes.c_int32),
        ("freq", ctypes.c_void_p),
        ("axis", ctypes.c_void_p),
    ]


class convrot_heads(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("heads", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("batch_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


class convrot_moe_weights(ctypes.Structure):
    _fields_ = [
        ("magic", ctypes.c_uint32),
        ("version", ctypes.c_uint32),
        ("experts", ctypes.c_int32),
        ("shared", ctypes.c_int32),
        ("K", ctypes.c_int64),
        ("F", ctypes.c_int64),
        ("gate_up", ctypes.c_void_p),
        ("gate_up_scale", ctypes.c_void_p),
        ("down", ctypes.c_void_p),
        ("down_scale", ctypes.c_void_p),
    ]


_MW = ctypes.POINTER(convrot_moe_weights)
_FW = ctypes.POINTER(convrot_fp8_weights)
_RP = ctypes.POINTER(convrot_rope)
_H = ctypes.c_void_p         # const convrot_heads * (byref, or packed bytes)

_SIGNATURES = {
    "convrot_status_string": (ctypes.c_char_p, [_c_int]),
    "convrot_last_hip_error": (_c_int, []),
    "convrot_version": (_c_int, []),
    "convrot_weights_packed_bytes": (_c_sz, [_c_i64, _c_i64, _c_int]),
    "convrot_prepare_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_int, _c_int, _c_int]),
    "convrot_linear_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_int]),
    "lowrank_convrot_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int]),
    "convrot_mlp_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int]),
    "lowrank_convrot_padded_rank": (_c_i64, [_c_i64, _c_int]),
    "lowrank_convrot_prepare_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_int, _c_int]),
    "lowrank_convrot_prepare_weights": (
        _c_int, [_c_p, _c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _W, _W, _c_p, _c_sz, _c_p]),
    "convrot_linear_prepare_weights": (
        _c_int, [_c_p, _c_int, _c_int, _c_p, _c_i64, _c_i64, _c_int, _W, _c_p, _c_sz, _c_p]),
    "convrot_linear_forward": (
        _c_int, [_c_p, _c_i64, _W, _c_p, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_linear_forward_noalloc": (
        _c_int, [_c_p, _c_i64, _W, _c_p, _c_p, _c_int, _c_p]),
    "lowrank_convrot_forward": (
        _c_int, [_c_p, _c_i64, _W, _W, _c_p, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_mlp_forward": (
        _c_int, [_c_p, _c_i64, _W, _c_p, _W, _c_p, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_rotate_quantize": (
        _c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_int, ctypes.c_uint32, _c_p, _c_p, _c_p]),
    "convrot_gemm_i32": (_c_int, [_c_p, _c_i64, _W, _c_p, _c_p]),
    "convrot_gemm_dequant": (
        _c_int, [_c_p, _c_p, _c_i64, _W, _c_p, _c_p, _c_int, ctypes.c_uint32, _c_p]),
    "convrot_lowrank_factor1": (_c_int, [_c_p, _c_p, _c_i64, _W, _c_p, _c_p, _c_p]),
    "convrot_swiglu_prepare_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_int, _c_int]),
    "convrot_swiglu_prepare_weights": (
        _c_int, [_c_p, _c_int, _c_p, _c_i64, _c_i64, _c_int, _W, _c_p, _c_sz, _c_p]),
    "convrot_swiglu_mlp_workspace_bytes": (
        _c_sz, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_int]),
    "convrot_swiglu_mlp_forward": (
        _c_int, [_c_p, _c_i64, _W, _c_p, _W, _c_p, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_swiglu_bf16": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p]),
    "convrot_silu_f32": (_c_int, [_c_p, _c_i64, _c_p, _c_p]),
    "lowrank_bf16_workspace_bytes": (ctypes.c_size_t, [_c_i64, _c_i64]),
    "lowrank_bf16_forward": (
        _c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p,
                 ctypes.c_size_t, _c_p]),
    "convrot_gelu_bf16": (_c_int, [_c_p, _c_i64, _c_p, _c_p]),
    "convrot_fp8_packed_bytes": (_c_sz, [_c_i64, _c_i64]),
    "convrot_fp8_scale_bytes": (_c_sz, [_c_i64, _c_i64]),
    "convrot_fp8_prepare_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_int, _c_int]),
    "convrot_fp8_linear_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "convrot_fp8_prepare_weights": (
        _c_int, [_c_p, _c_int, _c_int, _c_p, _c_i64, _c_i64, _FW, _c_p, _c_sz, _c_p]),
    "convrot_fp8_linear_forward": (
        _c_int, [_c_p, _c_i64, _FW, _c_p, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_fp8_quantize": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p]),
    "convrot_fp8_gemm_dequant": (
        _c_int, [_c_p, _c_p, _c_i64, _FW, _c_p, _c_p, _c_int, _c_p]),
    "convrot_fp8_gemm_dequant_scales": (
        _c_int, [_c_p, _c_p, _c_int, _c_i64, _FW, _c_p, _c_p, _c_int, _c_p]),
    "convrot_rope_prepare": (
        _c_int, [ctypes.POINTER(ctypes.c_int32), _c_int, _c_int, ctypes.c_double, _c_int, _c_int,
                 _RP, _c_p]),
    "convrot_rope_forward": (
        _c_int, [_c_i64, _c_i64, _c_int, _H, _H, _H, _H, _RP, _c_p, _c_int, _c_i64,
                 ctypes.c_uint32, _c_p]),
    "convrot_qk_norm_rope_forward": (
        _c_int, [_c_i64, _c_i64, _c_int, _H, _H, _c_p, _H, _H, _c_p, ctypes.c_float, _RP, _c_p,
                 _c_int, _c_i64, _c_p]),
    "convrot_qk_norm_rope_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_int, _c_int, _c_int]),
    "convrot_qk_norm_rope_backward": (
        _c_int, [_c_i64, _c_i64, _c_int, _H, _H, _H, _c_p, _c_p, _H, _H, _H, _c_p, _c_p,
                 ctypes.c_float, _RP, _c_p, _c_int, _c_i64, _c_p, _c_sz, _c_p]),
    "convrot_qkv_forward": (
        _c_int, [_c_p, _c_i64, _c_i64, _W, _c_p, _c_int, _c_int, _c_p, _c_p, ctypes.c_float, _RP,
                 _c_p, _c_int, _c_i64, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_fp8_qkv_forward": (
        _c_int, [_c_p, _c_i64, _c_i64, _FW, _c_p, _c_int, _c_int, _c_p, _c_p, ctypes.c_float, _RP,
                 _c_p, _c_int, _c_i64, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "convrot_add_rms_norm_forward": (
        _c_int, [_c_p, _c_int, _c_p, _c_int, _c_p, ctypes.c_float, _c_i64, _c_i64, _c_p, _c_p,
                 _c_int, _c_p]),
    "convrot_add_rms_norm_rotate_quantize": (
        _c_int, [_c_p, _c_int, _c_p, _c_int, _c_p, ctypes.c_float, _c_i64, _c_i64, _c_int,
                 ctypes.c_uint32, _c_p, _c_p, _c_p, _c_p]),
    "convrot_add_rms_norm_fp8_quantize": (
        _c_int, [_c_p, _c_int, _c_p, _c_int, _c_p, ctypes.c_float, _c_i64, _c_i64, _c_int, _c_p,
                 _c_p, _c_p, _c_p]),
    "convrot_fp8_norm_linear_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "convrot_norm_linear_forward": (
        _c_int, [_c_p, _c_int, _c_p, _c_int, _c_p, ctypes.c_float, _c_i64, _W, _c_p, _c_p, _c_p,
                 _c_int, _c_p, _c_sz, _c_p]),
    "convrot_fp8_norm_linear_forward": (
        _c_int, [_c_p, _c_int, _c_p, _c_int, _c_p, ctypes.c_float, _c_i64, _FW, _c_p, _c_p, _c_p,
                 _c_int, _c_p, _c_sz, _c_p]),
    "convrot_add_rms_norm_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "convrot_add_rms_norm_backward": (
        _c_int, [_c_p, _c_int, _c_p, _c_int, _c_p, _c_p, ctypes.c_float, _c_i64, _c_i64, _c_p,
                 _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "convrot_moe_packed_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "convrot_moe_scale_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "convrot_moe_prepare_weights": (
        _c_int, [_c_p, _c_p, _c_int, _c_p, _c_p, _c_int, _MW, _c_p]),
    "convrot_moe_workspace_bytes": (_c_sz, [_c_i64, _MW, _c_int]),
    "convrot_moe_forward": (
        _c_int, [_c_p, _c_i64, _c_p, _c_int, _c_p, _MW, _c_int, _c_int, ctypes.c_uint32,
                 ctypes.c_float, _c_p, _c_int, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "convrot_probe_mfma_i8": (_c_int, [_c_i64, _c_p, _c_p, ctypes.POINTER(ctypes.c_int64),
                                       _c_p]),
    "convrot_probe_stream": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_p]),
}

EXPORTED = tuple(_SIGNATURES)

_lib = None


class ConvRotError(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib = library()
        msg = lib.convrot_status_string(status).decode()
        extra = ""
        if status == EHIP:
            extra = f" (hipError {lib.convrot_last_hip_error()})"
        super().__init__(f"{fn} failed: {msg} [{status}]{extra}")
        self.status = status


def library():
    """Load libconvrot.so (built in-tree by ``w8a8_int8_rotated_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m w8a8_int8_rotated_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(fn: str, rc: int):
    if rc != OK:
        raise ConvRotError(fn, rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _launch(device, fn: str, *args):
    """Call the library with `device` current, on that device's current stream."""
    index = device.index
    # the raw handle: a Stream object costs as much as the launch's checks
    raw = torch._C._cuda_getCurrentRawStream(index)
    fun = getattr(_lib or library(), fn)
    if index == torch.cuda.current_device():
        rc = fun(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fun(*args, raw)
    if rc:
        _check(fn, rc)


def _tensors(v):
    """The tensors an argument or a result consists of."""
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, tuple):
        for x in v:
            yield from _tensors(x)
    elif isinstance(v, (PreparedWeights, FP8Weights, RopePlan, MoEWeights)):
        yield from (t for t in vars(v).values() if isinstance(t, torch.Tensor))


def _on_stream(fn, args: dict):
    """fn(**args) on args["stream"], which must be ordered after whatever made the
    arguments.  It is the current stream for the whole call, so that what the call
    copies, reads back and allocates is ordered on it too; nothing of the call is
    ordered against the stream that was current.  The allocator keeps the arguments'
    memory until this stream has passed the call, and the results' (this stream's)
    until the stream that was current has passed what it uses them for."""
    stream = args.pop("stream")
    device = args.get("device")
    if device is not None and torch.device(device).index not in (None, stream.device.index):
        raise ValueError(f"stream is on {stream.device}, device is {device}")
    _on_device(stream.device,
               **{n: t for n, t in args.items() if isinstance(t, torch.Tensor)})
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return fn(**args)
    with torch.cuda.stream(stream):
        out = fn(**args)
    for t in _tensors(tuple(args.values())):
        t.record_stream(stream)
    for t in _tensors(out if isinstance(out, tuple) else (out,)):
        t.record_stream(current)
    return out


_DTYPE_TAGS = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8, torch.int32: I32,
               torch.float8_e4m3fn: F8E4M3}


def _dtype_tag(dt: torch.dtype) -> int:
    return _DTYPE_TAGS[dt]


def _torch_dtype(tag: int) -> torch.dtype:
    return {F32: torch.float32, BF16: torch.bfloat16}[tag]


def _on_device(device, **tensors):
    """Every tensor the library will dereference is a GPU tensor on `device`
    (any GPU when None).  Called after the shape and dtype checks, so a
    host-side caller sees those errors first."""
    if device is not None and device.type == "cuda":
        for t in tensors.values():
            if t is not None and t.device != device:
                break
        else:
            return
    for name, t in tensors.items():
        if t is None:
            continue
        d = t.device
        if d.type != "cuda" or (device is not None and d != device):
            raise ValueError(f"{name} must be a GPU tensor on {device or 'the GPU'}, got {d}")


def _need(t, name: str, dtypes, shape):
    """Check a tensor argument before its pointer reaches the library: its
    dtype, exact shape and contiguity (the device is checked by _on_device)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _opt(t, name: str, dtypes, shape):
    return None if t is None else _need(t, name, dtypes, shape)


def _weights(W, name: str):
    if not isinstance(W, PreparedWeights):
        raise ValueError(f"{name} must be PreparedWeights from convrot_linear_prepare_weights")
    return W.codes.device


def _rows(X, name: str, K: int):
    """bf16 activations [M, K]; returns M."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor [M, {K}]")
    _need(X, name, torch.bfloat16, (X.shape[0], K))
    return X.shape[0]


def _output(out, M: int, N: int, dtypes):
    return None if out is None else _need(out, "out", dtypes, (M, N))


def _check_workspace(nbytes: int, workspace):
    if workspace is None or nbytes == 0:
        return
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 \
            or workspace.dim() != 1 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    if workspace.numel() < nbytes:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, {nbytes} needed")


def _workspace(nbytes: int, device, workspace):
    if nbytes == 0:
        return None
    if workspace is not None:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------- sizing ----

def convrot_weights_packed_bytes(N: int, K: int, block: int) -> int:
    return library().convrot_weights_packed_bytes(N, K, block)


def convrot_prepare_workspace_bytes(N, K, block, w_dtype, layout) -> int:
    return library().convrot_prepare_workspace_bytes(N, K, block, w_dtype, layout)


def convrot_linear_workspace_bytes(M, K, N, block) -> int:
    return library().convrot_linear_workspace_bytes(M, K, N, block)


def lowrank_convrot_workspace_bytes(M, K, r, N, block) -> int:
    return library().lowrank_convrot_workspace_bytes(M, K, r, N, block)


def convrot_mlp_workspace_bytes(M, K, F, N, block) -> int:
    return library().convrot_mlp_workspace_bytes(M, K, F, N, block)


def lowrank_bf16_workspace_bytes(M, r) -> int:
    return library().lowrank_bf16_workspace_bytes(M, r)


# ----------------------------------------------------------- weights ----

class PreparedWeights:
    """A prepared weight: the C descriptor plus the tensors it points into."""

    def __init__(self, desc: convrot_weights, codes: torch.Tensor, scale: torch.Tensor):
        self.desc = desc
        self.codes = codes
        self.scale = scale

    @property
    def N(self):
        return self.desc.N

    @property
    def K(self):
        return self.desc.K

    @property
    def block(self):
        return self.desc.block

    def ref(self):
        return ctypes.byref(self.desc)


def convrot_linear_prepare_weights(W: torch.Tensor, block: int, layout: int = OUT_MAJOR,
                                   src_scale: torch.Tensor | None = None,
                                   stream=None, rotation: str = "sylvester") -> PreparedWeights:
    """Rotate + quantise + pack a weight (``[N, K]`` or ``[K, N]`` per layout)
    with the rotation kind ``'sylvester'`` or ``'regular'``."""
    if stream is not None:
        return _on_stream(convrot_linear_prepare_weights, locals())
    lib = library()
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a 2-D tensor")
    if layout not in (OUT_MAJOR, IN_MAJOR):
        raise ValueError("layout must be OUT_MAJOR or IN_MAJOR")
    if layout == OUT_MAJOR:
        N, K = W.shape
    else:
        K, N = W.shape
    if W.dtype not in (torch.float32, torch.bfloat16, torch.int8):
        raise ValueError(f"W must be float32, bfloat16 or int8 codes, got {W.dtype}")
    if (W.dtype == torch.int8) != (src_scale is not None):
        raise ValueError("src_scale is required for int8 codes and only for them")
    _opt(src_scale, "src_scale", torch.float32, (N,))
    if rotation not in ROTATIONS:
        raise ValueError(f"rotation must be one of {sorted(ROTATIONS)}")
    W = W.contiguous()
    _on_device(W.device, W=W, src_scale=src_scale)
    tag = _dtype_tag(W.dtype)
    nbytes = lib.convrot_weights_packed_bytes(N, K, block)
    if nbytes == 0:
        raise ConvRotError("convrot_linear_prepare_weights", EUNSUPPORTED)
    codes = torch.empty(nbytes, dtype=torch.int8, device=W.device)
    scale = torch.empty(N, dtype=torch.float32, device=W.device)
    desc = convrot_weights()
    desc.codes = codes.data_ptr()
    desc.scale = scale.data_ptr()
    desc.flags = ROTATIONS[rotation]
    wsb = lib.convrot_prepare_workspace_bytes(N, K, block, tag, layout)
    ws = _workspace(wsb, W.device, None)
    rc = lib.convrot_linear_prepare_weights(
        _ptr(W), tag, layout, _ptr(src_scale), N, K, block, ctypes.byref(desc), _ptr(ws),
        wsb, _stream(stream))
    _check("convrot_linear_prepare_weights", rc)
    pw = PreparedWeights(desc, codes, scale)
    pw._ws = ws  # keep alive until the stream has consumed it
    return pw


def lowrank_padded_rank(r: int, block: int) -> int:
    """The rank a low-rank pair is stored with (lowrank_convrot_padded_rank)."""
    return library().lowrank_convrot_padded_rank(r, block)


def convrot_lowrank_prepare(A: torch.Tensor, B: torch.Tensor, block: int, stream=None,
                            rotation: str = "sylvester"):
    """Prepare a low-rank pair W ~ B . A, A [r, K] and B [N, r] (output-major,
    float32 or bfloat16) with lowrank_convrot_prepare_weights, which pads the
    rank with zero rows of A and zero columns of B to
    lowrank_padded_rank(r, block).  Returns two PreparedWeights."""
    if stream is not None:
        return _on_stream(convrot_lowrank_prepare, locals())
    lib = library()
    for t, name in ((A, "A"), (B, "B")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D tensor")
    r, K = A.shape
    N = B.shape[0]
    if A.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"A must be float32 or bfloat16, got {A.dtype}")
    B = B.contiguous()
    _need(B, "B", A.dtype, (N, r))
    if rotation not in ROTATIONS:
        raise ValueError(f"rotation must be one of {sorted(ROTATIONS)}")
    A = A.contiguous()
    _on_device(A.device, A=A, B=B)
    tag = _dtype_tag(A.dtype)
    rp = lib.lowrank_convrot_padded_rank(r, block)
    na, nb = lib.convrot_weights_packed_bytes(rp, K, block), lib.convrot_weights_packed_bytes(N, rp, block)
    if rp == 0 or na == 0 or nb == 0:
        raise ConvRotError("lowrank_convrot_prepare_weights", EUNSUPPORTED)
    dev = A.device
    pws = []
    descs = []
    for n, nbytes in ((rp, na), (N, nb)):
        d = convrot_weights()
        codes = torch.empty(nbytes, dtype=torch.int8, device=dev)
        scale = torch.empty(n, dtype=torch.float32, device=dev)
        d.codes, d.scale, d.flags = codes.data_ptr(), scale.data_ptr(), ROTATIONS[rotation]
        descs.append(d)
        pws.append((codes, scale))
    wsb = lib.lowrank_convrot_prepare_workspace_bytes(r, K, N, block, tag)
    ws = _workspace(wsb, dev, None)
    rc = lib.lowrank_convrot_prepare_weights(
        _ptr(A), _ptr(B), tag, r, K, N, block, ctypes.byref(descs[0]), ctypes.byref(descs[1]),
        _ptr(ws), wsb, _stream(stream))
    _check("lowrank_convrot_prepare_weights", rc)
    pa = PreparedWeights(descs[0], *pws[0])
    pb = PreparedWeights(descs[1], *pws[1])
    pa._ws = pb._ws = ws    # keep alive until the stream has consumed it
    return pa, pb


# ----------------------------------------------------------- forward ----

def convrot_linear_forward(X: torch.Tensor, W: PreparedWeights, bias=None,
                           out_dtype: torch.dtype = torch.bfloat16, out=None,
                           workspace=None, stream=None) -> torch.Tensor:
    if stream is not None:
        return _on_stream(convrot_linear_forward, locals())
    lib = library()
    dev = _weights(W, "W")
    M = _rows(X, "X", W.K)
    _opt(bias, "bias", torch.float32, (W.N,))
    _output(out, M, W.N, (torch.bfloat16, torch.float32))
    wsb = lib.convrot_linear_workspace_bytes(M, W.K, W.N, W.block)
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, bias=bias, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, W.N), dtype=out_dtype, device=dev)
    ws = _workspace(wsb, dev, workspace)
    rc = lib.convrot_linear_forward(_ptr(X), M, W.ref(), _ptr(bias), _ptr(out),
                                    _dtype_tag(out.dtype), _ptr(ws),
                                    ws.numel() if ws is not None else 0, _stream(stream))
    _check("convrot_linear_forward", rc)
    return out


def convrot_linear_forward_noalloc(X: torch.Tensor, W: PreparedWeights, bias=None,
                                   out_dtype: torch.dtype = torch.bfloat16, out=None,
                                   stream=None) -> torch.Tensor:
    """convrot_linear_forward with the library's static device scratch as its
    workspace (the C call allocates nothing; pass `out` to allocate nothing
    here either).  Calls on one device must not overlap in time."""
    if stream is not None:
        return _on_stream(convrot_linear_forward_noalloc, locals())
    lib = library()
    dev = _weights(W, "W")
    M = _rows(X, "X", W.K)
    _opt(bias, "bias", torch.float32, (W.N,))
    _output(out, M, W.N, (torch.bfloat16, torch.float32))
    _on_device(dev, X=X, bias=bias, out=out)
    if out is None:
        out = torch.empty((M, W.N), dtype=out_dtype, device=dev)
    rc = lib.convrot_linear_forward_noalloc(_ptr(X), M, W.ref(), _ptr(bias), _ptr(out),
                                            _dtype_tag(out.dtype), _stream(stream))
    _check("convrot_linear_forward_noalloc", rc)
    return out


def lowrank_convrot_forward(X: torch.Tensor, A: PreparedWeights, B: PreparedWeights,
                            bias=None, out_dtype: torch.dtype = torch.bfloat16, out=None,
                            workspace=None, stream=None) -> torch.Tensor:
    if stream is not None:
        return _on_stream(lowrank_convrot_forward, locals())
    lib = library()
    dev = _weights(A, "A")
    if _weights(B, "B") != dev:
        raise ValueError("A and B must be on the same device")
    M = _rows(X, "X", A.K)
    _opt(bias, "bias", torch.float32, (B.N,))
    _output(out, M, B.N, (torch.bfloat16, torch.float32))
    wsb = lib.lowrank_convrot_workspace_bytes(M, A.K, A.N, B.N, A.block)
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, bias=bias, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, B.N), dtype=out_dtype, device=dev)
    ws = _workspace(wsb, dev, workspace)
    rc = lib.lowrank_convrot_forward(_ptr(X), M, A.ref(), B.ref(), _ptr(bias), _ptr(out),
                                     _dtype_tag(out.dtype), _ptr(ws),
                                     ws.numel() if ws is not None else 0, _stream(stream))
    _check("lowrank_convrot_forward", rc)
    return out


def convrot_mlp_forward(X: torch.Tensor, W_up: PreparedWeights, W_down: PreparedWeights,
                        bias_up=None, bias_down=None, out_dtype: torch.dtype = torch.bfloat16,
                        out=None, workspace=None, stream=None) -> torch.Tensor:
    if stream is not None:
        return _on_stream(convrot_mlp_forward, locals())
    lib = library()
    dev = _weights(W_up, "W_up")
    if _weights(W_down, "W_down") != dev:
        raise ValueError("W_up and W_down must be on the same device")
    M = _rows(X, "X", W_up.K)
    _opt(bias_up, "bias_up", torch.float32, (W_up.N,))
    _opt(bias_down, "bias_down", torch.float32, (W_down.N,))
    _output(out, M, W_down.N, (torch.bfloat16, torch.float32))
    wsb = lib.convrot_mlp_workspace_bytes(M, W_up.K, W_up.N, W_down.N, W_up.block)
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, bias_up=bias_up, bias_down=bias_down, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, W_down.N), dtype=out_dtype, device=dev)
    ws = _workspace(wsb, dev, workspace)
    rc = lib.convrot_mlp_forward(_ptr(X), M, W_up.ref(), _ptr(bias_up), W_down.ref(),
                                 _ptr(bias_down), _ptr(out), _dtype_tag(out.dtype), _ptr(ws),
                                 ws.numel() if ws is not None else 0, _stream(stream))
    _check("convrot_mlp_forward", rc)
    return out


# ------------------------------------------------------------ SwiGLU ----

def convrot_swiglu_mlp_workspace_bytes(M, K, F, N, block_up, block_down) -> int:
    return library().convrot_swiglu_mlp_workspace_bytes(M, K, F, N, block_up, block_down)


def convrot_swiglu_prepare(W: torch.Tensor, block: int, src_scale: torch.Tensor | None = None,
                           stream=None, rotation: str = "sylvester") -> PreparedWeights:
    """Prepare a SwiGLU fc1 weight [2F, K] (gate rows, then up rows): float32 or
    bfloat16 weights, or int8 codes with src_scale [2F]; stored interleaved
    (SWIGLU_PAIRS) for the fused SwiGLU epilogue."""
    if stream is not None:
        return _on_stream(convrot_swiglu_prepare, locals())
    lib = library()
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.shape[0] % 2:
        raise ValueError("W must be a 2-D tensor [2F, K]")
    N2, K = W.shape
    if W.dtype not in (torch.float32, torch.bfloat16, torch.int8):
        raise ValueError(f"W must be float32, bfloat16 or int8 codes, got {W.dtype}")
    if (W.dtype == torch.int8) != (src_scale is not None):
        raise ValueError("src_scale is required for int8 codes and only for them")
    _opt(src_scale, "src_scale", torch.float32, (N2,))
    if rotation not in ROTATIONS:
        raise ValueError(f"rotation must be one of {sorted(ROTATIONS)}")
    W = W.contiguous()
    _on_device(W.device, W=W, src_scale=src_scale)
    tag = _dtype_tag(W.dtype)
    nbytes = lib.convrot_weights_packed_bytes(N2, K, block)
    wsb = lib.convrot_swiglu_prepare_workspace_bytes(N2 // 2, K, block, tag)
    if nbytes == 0 or wsb == 0:
        raise ConvRotError("convrot_swiglu_prepare_weights", EUNSUPPORTED)
    codes = torch.empty(nbytes, dtype=torch.int8, device=W.device)
    scale = torch.empty(N2, dtype=torch.float32, device=W.device)
    desc = convrot_weights()
    desc.codes, desc.scale, desc.flags = codes.data_ptr(), scale.data_ptr(), ROTATIONS[rotation]
    ws = _workspace(wsb, W.device, None)
    rc = lib.convrot_swiglu_prepare_weights(_ptr(W), tag, _ptr(src_scale), N2 // 2, K, block,
                                            ctypes.byref(desc), _ptr(ws), wsb, _stream(stream))
    _check("convrot_swiglu_prepare_weights", rc)
    pw = PreparedWeights(desc, codes, scale)
    pw._ws = ws
    return pw


def convrot_swiglu_mlp_forward(X: torch.Tensor, W_gu: PreparedWeights, W_down: PreparedWeights,
                               bias_gu=None, bias_down=None,
                               out_dtype: torch.dtype = torch.bfloat16, out=None,
                               workspace=None, stream=None) -> torch.Tensor:
    """Y = linear(swiglu(linear(X; W_gu) + bias_gu); W_down) + bias_down."""
    if stream is not None:
        return _on_stream(convrot_swiglu_mlp_forward, locals())
    lib = library()
    dev = _weights(W_gu, "W_gu")
    if _weights(W_down, "W_down") != dev:
        raise ValueError("W_gu and W_down must be on the same device")
    M = _rows(X, "X", W_gu.K)
    F = W_down.K
    _opt(bias_gu, "bias_gu", torch.float32, (W_gu.N,))
    _opt(bias_down, "bias_down", torch.float32, (W_down.N,))
    _output(out, M, W_down.N, (torch.bfloat16, torch.float32))
    wsb = lib.convrot_swiglu_mlp_workspace_bytes(M, W_gu.K, F, W_down.N, W_gu.block,
                                                 W_down.block)
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, bias_gu=bias_gu, bias_down=bias_down, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, W_down.N), dtype=out_dtype, device=dev)
    ws = _workspace(wsb, dev, workspace)
    rc = lib.convrot_swiglu_mlp_forward(_ptr(X), M, W_gu.ref(), _ptr(bias_gu), W_down.ref(),
                                        _ptr(bias_down), _ptr(out), _dtype_tag(out.dtype),
                                        _ptr(ws), ws.numel() if ws is not None else 0,
                                        _stream(stream))
    _check("convrot_swiglu_mlp_forward", rc)
    return out


def convrot_swiglu_bf16(gu: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """g [M, F] = bf16(fp32(silu(gate)) * up) for gu [M, 2F] = gate | up."""
    if stream is not None:
        return _on_stream(convrot_swiglu_bf16, locals())
    lib = library()
    if not isinstance(gu, torch.Tensor) or gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError("gu must be a 2-D tensor [M, 2F]")
    M, F = gu.shape[0], gu.shape[1] // 2
    _need(gu, "gu", torch.bfloat16, (M, 2 * F))
    _opt(out, "out", torch.bfloat16, (M, F))
    _on_device(gu.device, gu=gu, out=out)
    if out is None:
        out = torch.empty((M, F), dtype=torch.bfloat16, device=gu.device)
    _check("convrot_swiglu_bf16", lib.convrot_swiglu_bf16(_ptr(gu), M, F, _ptr(out),
                                                          _stream(stream)))
    return out


def convrot_silu_f32(a: torch.Tensor, stream=None) -> torch.Tensor:
    """fp32(silu(a)) of bf16 values, as every SwiGLU path computes it."""
    if stream is not None:
        return _on_stream(convrot_silu_f32, locals())
    lib = library()
    if not isinstance(a, torch.Tensor) or a.dtype != torch.bfloat16:
        raise ValueError("a must be a bf16 tensor")
    a = a.contiguous()
    _on_device(a.device, a=a)
    out = torch.empty(a.shape, dtype=torch.float32, device=a.device)
    _check("convrot_silu_f32", lib.convrot_silu_f32(_ptr(a), a.numel(), _ptr(out),
                                                    _stream(stream)))
    return out


def lowrank_bf16_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, bias=None,
                         out=None, workspace=None, stream=None) -> torch.Tensor:
    """Comparison variant: bf16(bf16(X . A^T) . B^T + bias), bf16 factors
    A [r, K] and B [N, r], no rotation or quantisation."""
    if stream is not None:
        return _on_stream(lowrank_bf16_forward, locals())
    lib = library()
    for t, name in ((X, "X"), (A, "A"), (B, "B")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D tensor")
    M, K = X.shape
    r, N = A.shape[0], B.shape[0]
    dev = A.device
    _need(X, "X", torch.bfloat16, (M, K))
    _need(A, "A", torch.bfloat16, (r, K))
    _need(B, "B", torch.bfloat16, (N, r))
    _opt(bias, "bias", torch.float32, (N,))
    _output(out, M, N, torch.bfloat16)
    wsb = lib.lowrank_bf16_workspace_bytes(M, r)
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, A=A, B=B, bias=bias, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ws = _workspace(wsb, dev, workspace)
    rc = lib.lowrank_bf16_forward(_ptr(X), M, K, _ptr(A), r, _ptr(B), N, _ptr(bias), _ptr(out),
                                  _ptr(ws), ws.numel() if ws is not None else 0,
                                  _stream(stream))
    _check("lowrank_bf16_forward", rc)
    return out


# --------------------------------------------- FP8 block-scaled linear ----

class FP8Weights:
    """A prepared FP8 weight: the C descriptor plus the tensors it points into."""

    def __init__(self, desc: convrot_fp8_weights, codes: torch.Tensor, scale: torch.Tensor):
        self.desc = desc
        self.codes = codes
        self.scale = scale
        self._ref = ctypes.byref(desc)

    @property
    def N(self):
        return self.desc.N

    @property
    def K(self):
        return self.desc.K

    def ref(self):
        return self._ref


def _fp8_weights(W, name: str):
    if not isinstance(W, FP8Weights):
        raise ValueError(f"{name} must be FP8Weights from convrot_fp8_prepare_weights")
    return W.codes.device


def convrot_fp8_packed_bytes(N: int, K: int) -> int:
    return library().convrot_fp8_packed_bytes(N, K)


def convrot_fp8_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    return library().convrot_fp8_linear_workspace_bytes(M, K, N)


def convrot_fp8_prepare_weights(W: torch.Tensor, layout: int = OUT_MAJOR,
                                src_scale: torch.Tensor | None = None, scales: str = "f32",
                                stream=None) -> FP8Weights:
    """Quantise and pack a weight (``[N, K]`` or ``[K, N]`` per layout) to e4m3
    with one scale per 128 x 128 block, float32 or (scales='pow2') a power of
    two; or import float8_e4m3fn codes with src_scale [ceil(N/128), K/128]."""
    if stream is not None:
        return _on_stream(convrot_fp8_prepare_weights, locals())
    lib = library()
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a 2-D tensor")
    if layout not in (OUT_MAJOR, IN_MAJOR):
        raise ValueError("layout must be OUT_MAJOR or IN_MAJOR")
    N, K = W.shape if layout == OUT_MAJOR else W.shape[::-1]
    if W.dtype not in (torch.float32, torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"W must be float32, bfloat16 or float8_e4m3fn codes, got {W.dtype}")
    if (W.dtype == torch.float8_e4m3fn) != (src_scale is not None):
        raise ValueError("src_scale is required for float8_e4m3fn codes and only for them")
    _opt(src_scale, "src_scale", torch.float32, (-(-N // 128), K // 128))
    if scales not in FP8_SCALES:
        raise ValueError(f"scales must be one of {sorted(FP8_SCALES)}")
    nbytes = lib.convrot_fp8_packed_bytes(N, K)
    if nbytes == 0:
        raise ConvRotError("convrot_fp8_prepare_weights", EUNSUPPORTED)
    W = W.contiguous()
    _on_device(W.device, W=W, src_scale=src_scale)
    if src_scale is not None and scales == "pow2":
        # load time: the one check that reads the tensors' values
        bits = src_scale.view(torch.int32)
        if bool((((bits & 0x7FFFFF) != 0) | (bits < 0) | (bits == 0x7F800000)).any()):
            raise ValueError("src_scale of a pow2 weight must hold powers of two or zeros")
        if bool((bits == 0).any()):
            # the matrix instruction reads a zero as 2^-127
            c = W if layout == OUT_MAJOR else W.t()
            used = torch.nn.functional.pad((c.view(torch.uint8) & 0x7F) != 0, (0, 0, 0, -N % 128))
            used = used.view(-(-N // 128), 128, K // 128, 128).any(3).any(1)
            if bool((used & (bits == 0)).any()):
                raise ValueError("a block whose scale is 0 must hold zero codes")
    tag = _dtype_tag(W.dtype)
    codes = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    scale = torch.empty((-(-N // 128), K // 128), dtype=torch.float32, device=W.device)
    desc = convrot_fp8_weights()
    desc.codes, desc.scale, desc.scales = codes.data_ptr(), scale.data_ptr(), FP8_SCALES[scales]
    wsb = lib.convrot_fp8_prepare_workspace_bytes(N, K, tag, layout)
    ws = _workspace(wsb, W.device, None)
    _launch(W.device, "convrot_fp8_prepare_weights", _ptr(W), tag, layout,
            _ptr(src_scale), N, K, ctypes.byref(desc), _ptr(ws), wsb)
    fw = FP8Weights(desc, codes, scale)
    fw._ws = ws  # keep alive until the stream has consumed it
    return fw


def convrot_fp8_linear_forward(X: torch.Tensor, W: FP8Weights, bias=None,
                               out_dtype: torch.dtype = torch.bfloat16, out=None,
                               workspace=None, stream=None) -> torch.Tensor:
    """Y [M, N] = X . W^T (+ bias) with X quantised to e4m3 per 128 inputs."""
    if stream is not None:
        return _on_stream(convrot_fp8_linear_forward, locals())
    lib = library()
    dev = _fp8_weights(W, "W")
    M = _rows(X, "X", W.K)
    _opt(bias, "bias", torch.float32, (W.N,))
    _output(out, M, W.N, (torch.bfloat16, torch.float32))
    wsb = lib.convrot_fp8_linear_workspace_bytes(M, W.K, W.N)
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, bias=bias, out=out, workspace=workspace)
    if out is None:
        out = torch.empty((M, W.N), dtype=out_dtype, device=dev)
    ws = _workspace(wsb, dev, workspace)
    _launch(dev, "convrot_fp8_linear_forward", _ptr(X), M, W.ref(), _ptr(bias),
            _ptr(out), _dtype_tag(out.dtype), _ptr(ws), ws.numel() if ws is not None else 0)
    return out


# ----------------------------------- norms and rotary positions of Q and K ----

class RopePlan:
    """A rotary plan: the C descriptor plus its tables.  freq (float64, radians
    per position unit) and axis (int32), one entry per pair, may be overwritten
    by a caller with other frequencies or another assignment of axes."""

    def __init__(self, desc: convrot_rope, freq: torch.Tensor, axis: torch.Tensor):
        self.desc = desc
        self.freq = freq
        self.axis = axis
        self._ref = ctypes.byref(desc)

    @property
    def axes(self):
        return self.desc.axes

    @property
    def head_dim(self):
        return self.desc.head_dim

    def ref(self):
        return self._ref


def convrot_rope_prepare(dims, head_dim: int, theta: float = 10000.0,
                         pairing: str = "interleaved", spectrum: str = "axis", device="cuda",
                         stream=None) -> RopePlan:
    """A plan whose axis a turns dims[a] channels of every head (1 to 4 axes,
    each even; together at most head_dim): pairs 'interleaved' (2p, 2p + 1) or
    'half' (p, p + R/2), every axis running through all frequencies
    (spectrum='axis') or the pairs sharing one spectrum ('whole')."""
    if stream is not None:
        return _on_stream(convrot_rope_prepare, locals())
    dims = [int(d) for d in dims]
    if not 1 <= len(dims) <= ROPE_MAX_AXES or any(d <= 0 or d % 2 for d in dims):
        raise ValueError(f"dims must be 1 to {ROPE_MAX_AXES} positive even numbers, got {dims}")
    if sum(dims) > head_dim:
        raise ValueError(f"dims {dims} exceed head_dim {head_dim}")
    if pairing not in ROPE_PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(ROPE_PAIRINGS)}")
    if spectrum not in ROPE_SPECTRA:
        raise ValueError(f"spectrum must be one of {sorted(ROPE_SPECTRA)}")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"device must be a GPU, got {device}")
    half = sum(dims) // 2
    freq = torch.empty(half, dtype=torch.float64, device=device)
    axis = torch.empty(half, dtype=torch.int32, device=device)
    desc = convrot_rope()
    desc.freq, desc.axis = freq.data_ptr(), axis.data_ptr()
    _launch(freq.device, "convrot_rope_prepare", (ctypes.c_int32 * len(dims))(*dims),
            len(dims), head_dim, theta, ROPE_PAIRINGS[pairing], ROPE_SPECTRA[spectrum],
            ctypes.byref(desc))
    return RopePlan(desc, freq, axis)


# convrot_heads, laid out by struct: several times cheaper to fill per call than
# a ctypes structure (a bytes object passes as the pointer)
_HEADS = struct.Struct("Piiqqq")
_pack_heads = _HEADS.pack
_Tensor = torch.Tensor
assert _HEADS.size == ctypes.sizeof(convrot_heads)


def _heads(t, name: str, dtype, dims: int, B: int, T: int, H, D: int) -> bytes:
    """The C view of a tensor of per-head rows [B, T, H, D], or with dims == 3
    [T, H, D] (H None: any); any strides with contiguous channels."""
    if not isinstance(t, _Tensor) or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} tensor")
    shape, st = t.shape, t.stride()
    if len(st) != dims:
        raise ValueError(f"{name} must have as many dimensions as q")
    if dims == 4:
        b, n, h, d = shape
        sb, sn, sh, sd = st
    else:
        n, h, d = shape
        sn, sh, sd = st
        b, sb = B, 0
    if d != D or n != T or b != B or (H is not None and h != H):
        want = (*((B,) if dims == 4 else ()), T, "heads" if H is None else H, D)
        raise ValueError(f"{name} must have shape {want}, got {tuple(shape)}")
    if sd != 1:
        raise ValueError(f"{name} must have contiguous channels")
    return _pack_heads(t.data_ptr(), h, 0, sb, sn, sh)


def _heads_pair(q, k, rope, positions):
    """The checks shared by the rope and norm calls: the leading dimensions
    (dims, B, T), the batch stride of the positions and the views of q and k
    (None without k)."""
    if not isinstance(rope, RopePlan):
        raise ValueError("rope must be a RopePlan from convrot_rope_prepare")
    if not isinstance(q, _Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be a tensor [B, T, heads, D] or [T, heads, D]")
    dtype = q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float32:
        raise ValueError(f"q must be float32 or bfloat16, got {dtype}")
    shape, D = q.shape, rope.desc.head_dim
    dims = len(shape)
    lead = (dims, shape[0] if dims == 4 else 1, shape[-3])
    vq = _heads(q, "q", dtype, *lead, None, D)
    vk = None if k is None else _heads(k, "k", dtype, *lead, None, D)
    return lead, _positions(positions, lead[1], lead[2], rope.desc.axes), vq, vk


def _positions(positions, B, T, axes):
    """The batch stride of checked positions."""
    if not isinstance(positions, _Tensor) \
            or (positions.dtype != torch.int32 and positions.dtype != torch.float32):
        raise ValueError("positions must be an int32 or float32 tensor")
    shape = positions.shape
    if not (shape == (T, axes) or shape == (B, T, axes)
            or (axes == 1 and shape in ((T,), (B, T)))):
        raise ValueError(f"positions must have shape {(T, axes)} or {(B, T, axes)}, got "
                         f"{tuple(shape)}")
    if not positions.is_contiguous():
        raise ValueError("positions must be contiguous")
    return T * axes if positions.numel() == B * T * axes else 0


def _heads_out(out, name, like, lead):
    """A caller's output, checked, or a new contiguous one, and its view."""
    if like is None:
        if out is not None:
            raise ValueError(f"{name} given without its input")
        return None, None
    shape = like.shape
    H, D = shape[-2], shape[-1]
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        HD = H * D
        return out, _pack_heads(out.data_ptr(), H, 0, lead[2] * HD, HD, D)
    return out, _heads(out, name, like.dtype, *lead, H, D)


def convrot_rope_forward(q: torch.Tensor, k, rope: RopePlan, positions: torch.Tensor,
                         inverse: bool = False, out_q=None, out_k=None, stream=None):
    """(q_out, k_out): q and k [B, T, heads, D] turned by the tokens' positions
    [T, axes] or [B, T, axes] (contiguous, int32 or float32); k may be None.  Out of
    place unless out_q is q.  inverse: by the negative angles, the backward pass
    (no autograd graph is built)."""
    if stream is not None:
        return _on_stream(convrot_rope_forward, locals())
    lead, psb, vq, vk = _heads_pair(q, k, rope, positions)
    _, B, T = lead
    dev = rope.freq.device
    _on_device(dev, q=q, k=k, positions=positions, out_q=out_q, out_k=out_k)
    out_q, oq = _heads_out(out_q, "out_q", q, lead)
    out_k, ok = _heads_out(out_k, "out_k", k, lead)
    _launch(dev, "convrot_rope_forward", B, T, _dtype_tag(q.dtype), vq, oq, vk, ok,
            rope.ref(), _ptr(positions), _dtype_tag(positions.dtype), psb,
            ROPE_INVERSE if inverse else 0)
    return out_q, out_k


def convrot_qk_norm_rope_forward(q: torch.Tensor, k, w_q, w_k, rope: RopePlan,
                                 positions: torch.Tensor, eps: float = 1e-6, out_q=None,
                                 out_k=None, stream=None):
    """convrot_rope_forward of q * rsqrt(mean(q^2) + eps) * w_q over each head's
    channels and of k likewise; w_q, w_k float32 [D] or None.  No autograd graph is
    built: convrot_qk_norm_rope_backward is the backward pass."""
    if stream is not None:
        return _on_stream(convrot_qk_norm_rope_forward, locals())
    lead, psb, vq, vk = _heads_pair(q, k, rope, positions)
    _, B, T = lead
    _opt(w_q, "w_q", torch.float32, (rope.head_dim,))
    _opt(w_k, "w_k", torch.float32, (rope.head_dim,))
    if k is None and w_k is not None:
        raise ValueError("w_k given without k")
    dev = rope.freq.device
    _on_device(dev, q=q, k=k, w_q=w_q, w_k=w_k, positions=positions, out_q=out_q, out_k=out_k)
    out_q, oq = _heads_out(out_q, "out_q", q, lead)
    out_k, ok = _heads_out(out_k, "out_k", k, lead)
    _launch(dev, "convrot_qk_norm_rope_forward", B, T, _dtype_tag(q.dtype), vq, oq,
            _ptr(w_q), vk, ok, _ptr(w_k), eps, rope.ref(), _ptr(positions),
            _dtype_tag(positions.dtype), psb)
    return out_q, out_k


def convrot_qk_norm_rope_workspace_bytes(B, T, heads_q, heads_k, head_dim) -> int:
    return library().convrot_qk_norm_rope_workspace_bytes(B, T, heads_q, heads_k, head_dim)


def convrot_qk_norm_rope_backward(g_q: torch.Tensor, g_k, q: torch.Tensor, k, w_q, w_k,
                                  rope: RopePlan, positions: torch.Tensor, eps: float = 1e-6,
                                  dq=None, dk=None, dw_q=None, dw_k=None, workspace=None,
                                  stream=None):
    """(dq, dk, dw_q, dw_k) of convrot_qk_norm_rope_forward(q, k, ...) from the
    gradients g_q and g_k of its outputs."""
    if stream is not None:
        return _on_stream(convrot_qk_norm_rope_backward, locals())
    lib = library()
    lead, psb, vq, vk = _heads_pair(q, k, rope, positions)
    _, B, T = lead
    D = rope.head_dim
    views = []
    for g, x, n in ((g_q, q, "g_q"), (g_k, k, "g_k")):
        if (g is None) != (x is None):
            raise ValueError(f"{n} must be given with its input and only then")
        views.append(None if g is None else _heads(g, n, x.dtype, *lead, x.shape[-2], D))
    if k is None and w_k is not None:
        raise ValueError("w_k given without k")
    if k is None and dw_k is not None:
        raise ValueError("dw_k given without k")
    for t, n in ((w_q, "w_q"), (w_k, "w_k"), (dw_q, "dw_q"), (dw_k, "dw_k")):
        _opt(t, n, torch.float32, (D,))
    wsb = lib.convrot_qk_norm_rope_workspace_bytes(B, T, q.shape[-2],
                                                   0 if k is None else k.shape[-2], D)
    _check_workspace(wsb, workspace)
    dev = rope.freq.device
    _on_device(dev, g_q=g_q, g_k=g_k, q=q, k=k, w_q=w_q, w_k=w_k, positions=positions, dq=dq,
               dk=dk, dw_q=dw_q, dw_k=dw_k, workspace=workspace)
    dq, vdq = _heads_out(dq, "dq", q, lead)
    dk, vdk = _heads_out(dk, "dk", k, lead)
    if dw_q is None:
        dw_q = torch.empty(D, dtype=torch.float32, device=dev)
    if dw_k is None and k is not None:
        dw_k = torch.empty(D, dtype=torch.float32, device=dev)
    ws = _workspace(wsb, dev, workspace)
    _launch(dev, "convrot_qk_norm_rope_backward", B, T, _dtype_tag(q.dtype), views[0],
            vq, vdq, _ptr(w_q), _ptr(dw_q), views[1], vk, vdk, _ptr(w_k), _ptr(dw_k), eps,
            rope.ref(), _ptr(positions), _dtype_tag(positions.dtype), psb, _ptr(ws),
            ws.numel() if ws is not None else 0)
    return dq, dk, dw_q, dw_k


def convrot_qkv_forward(X: torch.Tensor, W, heads_q: int, heads_kv: int, w_q, w_k,
                        rope: RopePlan, positions: torch.Tensor, bias=None, eps: float = 1e-6,
                        out_dtype: torch.dtype = torch.bfloat16, out=None, workspace=None,
                        stream=None) -> torch.Tensor:
    """The QKV projection of X [M, K] or [B, T, K] with the norms and rotation
    of its queries and keys: [.., (heads_q + 2 heads_kv) D], queries, keys, then
    values.  W: PreparedWeights or FP8Weights."""
    if stream is not None:
        return _on_stream(convrot_qkv_forward, locals())
    lib = library()
    fp8 = isinstance(W, FP8Weights)
    dev = _fp8_weights(W, "W") if fp8 else _weights(W, "W")
    if not isinstance(rope, RopePlan):
        raise ValueError("rope must be a RopePlan from convrot_rope_prepare")
    if not isinstance(X, torch.Tensor) or X.dim() not in (2, 3):
        raise ValueError(f"X must be a tensor [M, {W.K}] or [B, T, {W.K}]")
    _need(X, "X", torch.bfloat16, (*X.shape[:-1], W.K))
    B, T = (X.shape[0], X.shape[1]) if X.dim() == 3 else (1, X.shape[0])
    psb = _positions(positions, B, T, rope.axes)
    _opt(bias, "bias", torch.float32, (W.N,))
    _opt(w_q, "w_q", torch.float32, (rope.head_dim,))
    _opt(w_k, "w_k", torch.float32, (rope.head_dim,))
    _opt(out, "out", (torch.bfloat16, torch.float32), (*X.shape[:-1], W.N))
    M = B * T
    wsb = (lib.convrot_fp8_linear_workspace_bytes(M, W.K, W.N) if fp8 else
           lib.convrot_linear_workspace_bytes(M, W.K, W.N, W.block))
    _check_workspace(wsb, workspace)
    _on_device(dev, X=X, bias=bias, w_q=w_q, w_k=w_k, freq=rope.freq, positions=positions,
               out=out, workspace=workspace)
    if out is None:
        out = torch.empty((*X.shape[:-1], W.N), dtype=out_dtype, device=dev)
    ws = _workspace(wsb, dev, workspace)
    name = "convrot_fp8_qkv_forward" if fp8 else "convrot_qkv_forward"
    _launch(dev, name, _ptr(X), B, T, W.ref(), _ptr(bias), heads_q, heads_kv, _ptr(w_q),
            _ptr(w_k), eps, rope.ref(), _ptr(positions), _dtype_tag(positions.dtype), psb,
            _ptr(out), _dtype_tag(out.dtype), _ptr(ws), ws.numel() if ws is not None else 0)
    return out


# ------------------------- the residual's addition and the RMS norm ----

_FLOATS = (torch.bfloat16, torch.float32)


def _new(like: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """A new output of the contiguous `like`'s shape (empty_like is the cheaper call)."""
    if dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {dtype}")
    return torch.empty_like(like) if like.dtype == dtype else \
        torch.empty(like.shape, dtype=dtype, device=like.device)


def _gpu_of(t: torch.Tensor):
    """A tensor's device for _on_device; None, so that it refuses the tensor, off the GPU."""
    d = t.device
    return d if d.type == "cuda" else None


def _norm_args(x, w, residual, residual_out):
    """The checks the forward calls share: (M, K, the residual's dtype or x's)."""
    if not isinstance(x, _Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor [.., K]")
    shape = x.shape
    K = shape[-1]
    _need(x, "x", _FLOATS, shape)
    _opt(w, "w", torch.float32, (K,))
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out given without residual")
        return (x.numel() // K if K else 0), K, x.dtype
    _need(residual, "residual", _FLOATS, shape)
    if x.dtype == torch.float32 and residual.dtype != torch.float32:
        raise ValueError("a float32 x takes a float32 residual")
    _opt(residual_out, "residual_out", residual.dtype, shape)
    return (x.numel() // K if K else 0), K, residual.dtype


def convrot_add_rms_norm_forward(x: torch.Tensor, w, residual=None, eps: float = 1e-6,
                                 out_dtype: torch.dtype = torch.bfloat16, out=None,
                                 residual_out=None, stream=None):
    """(y, h): h = x + residual in the residual's type (None without a residual) and
    y = h * rsqrt(mean(h^2) + eps) * w over the last dimension; x and residual [.., K]
    contiguous, w float32 [K] or None.  residual_out may be residual itself.  No autograd
    graph is built: convrot_add_rms_norm_backward is the backward pass."""
    if stream is not None:
        return _on_stream(convrot_add_rms_norm_forward, locals())
    M, K, rdt = _norm_args(x, w, residual, residual_out)
    _opt(out, "out", _FLOATS, x.shape)
    dev = _gpu_of(x)
    _on_device(dev, x=x, w=w, residual=residual, out=out, residual_out=residual_out)
    if out is None:
        out = _new(x, out_dtype)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    _launch(dev, "convrot_add_rms_norm_forward", _ptr(x), _dtype_tag(x.dtype), _ptr(residual),
            _dtype_tag(rdt), _ptr(w), eps, M, K, _ptr(residual_out), _ptr(out),
            _dtype_tag(out.dtype))
    return out, residual_out


def convrot_add_rms_norm_rotate_quantize(x: torch.Tensor, w, block: int, residual=None,
                                         eps: float = 1e-6, rotation: str = "sylvester", q=None,
                                         s=None, residual_out=None, stream=None):
    """(q, s, h): the K-tiled INT8 codes (Mp, K) and row scales [M] of the rotated norm, as
    convrot_gemm_dequant takes them."""
    if stream is not None:
        return _on_stream(convrot_add_rms_norm_rotate_quantize, locals())
    M, K, rdt = _norm_args(x, w, residual, residual_out)
    q = _codes(q, M, K, x.device) if q is not None else None
    _opt(s, "s", torch.float32, (M,))
    if rotation not in ROTATIONS:
        raise ValueError(f"rotation must be one of {sorted(ROTATIONS)}")
    dev = _gpu_of(x)
    _on_device(dev, x=x, w=w, residual=residual, q=q, s=s, residual_out=residual_out)
    if q is None:
        q = _codes(None, M, K, dev)
    if s is None:
        s = torch.empty(M, dtype=torch.float32, device=dev)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    _launch(dev, "convrot_add_rms_norm_rotate_quantize", _ptr(x), _dtype_tag(x.dtype),
            _ptr(residual), _dtype_tag(rdt), _ptr(w), eps, M, K, block, ROTATIONS[rotation],
            _ptr(residual_out), _ptr(q), _ptr(s))
    return q, s, residual_out


def convrot_add_rms_norm_fp8_quantize(x: torch.Tensor, w, scales: str = "f32", residual=None,
                                      eps: float = 1e-6, q=None, s=None, residual_out=None,
                                      stream=None):
    """(q, s, h): the K-tiled e4m3 codes (Mp, K) and scales [K/128, Mp] of the norm, as
    convrot_fp8_gemm_dequant takes them."""
    if stream is not None:
        return _on_stream(convrot_add_rms_norm_fp8_quantize, locals())
    M, K, rdt = _norm_args(x, w, residual, residual_out)
    if scales not in FP8_SCALES:
        raise ValueError(f"scales must be one of {sorted(FP8_SCALES)}")
    Mp = padded_rows(M)
    _opt(q, "q", torch.uint8, (Mp, K))
    _opt(s, "s", torch.float32, (K // 128, Mp))
    dev = _gpu_of(x)
    _on_device(dev, x=x, w=w, residual=residual, q=q, s=s, residual_out=residual_out)
    if q is None:
        q = torch.empty((Mp, K), dtype=torch.uint8, device=dev)
    if s is None:
        s = torch.empty((K // 128, Mp), dtype=torch.float32, device=dev)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    _launch(dev, "convrot_add_rms_norm_fp8_quantize", _ptr(x), _dtype_tag(x.dtype),
            _ptr(residual), _dtype_tag(rdt), _ptr(w), eps, M, K, FP8_SCALES[scales],
            _ptr(residual_out), _ptr(q), _ptr(s))
    return q, s, residual_out


def convrot_fp8_norm_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    return library().convrot_fp8_norm_linear_workspace_bytes(M, K, N)


def convrot_norm_linear_forward(x: torch.Tensor, w, W, residual=None, bias=None,
                                eps: float = 1e-6, out_dtype: torch.dtype = torch.bfloat16,
                                out=None, residual_out=None, workspace=None, stream=None):
    """(Y, h): Y [.., N] = the linear W (PreparedWeights or FP8Weights) of the norm of
    h = x + residual, quantised as it is formed."""
    if stream is not None:
        return _on_stream(convrot_norm_linear_forward, locals())
    lib = library()
    fp8 = isinstance(W, FP8Weights)
    dev = _fp8_weights(W, "W") if fp8 else _weights(W, "W")
    M, K, rdt = _norm_args(x, w, residual, residual_out)
    if K != W.K:
        raise ValueError(f"x must have {W.K} channels, got {K}")
    shape = (*x.shape[:-1], W.N)
    _opt(bias, "bias", torch.float32, (W.N,))
    _opt(out, "out", _FLOATS, shape)
    wsb = (lib.convrot_fp8_norm_linear_workspace_bytes(M, K, W.N) if fp8 else
           lib.convrot_linear_workspace_bytes(M, K, W.N, W.block))
    _check_workspace(wsb, workspace)
    _on_device(dev, x=x, w=w, residual=residual, bias=bias, out=out, residual_out=residual_out,
               workspace=workspace)
    if out is None:
        if out_dtype not in _FLOATS:
            raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    ws = _workspace(wsb, dev, workspace)
    _launch(dev, "convrot_fp8_norm_linear_forward" if fp8 else "convrot_norm_linear_forward",
            _ptr(x), _dtype_tag(x.dtype), _ptr(residual), _dtype_tag(rdt), _ptr(w), eps, M,
            W.ref(), _ptr(bias), _ptr(residual_out), _ptr(out), _dtype_tag(out.dtype), _ptr(ws),
            ws.numel() if ws is not None else 0)
    return out, residual_out


def convrot_add_rms_norm_workspace_bytes(M: int, K: int) -> int:
    return library().convrot_add_rms_norm_workspace_bytes(M, K)


def convrot_add_rms_norm_backward(g: torch.Tensor, h: torch.Tensor, w, g_h=None,
                                  eps: float = 1e-6, x_dtype=None, dh=None, dx=None, dw=None,
                                  workspace=None, stream=None):
    """(dh, dx, dw) of convrot_add_rms_norm_forward from g, the gradient of y, and g_h, the
    gradient that reaches h otherwise (or None).  dh is the residual's gradient, in h's type;
    dx is x's: dh itself, or with x_dtype=torch.bfloat16 beside a float32 h its bf16 copy.
    dw is None without w."""
    if stream is not None:
        return _on_stream(convrot_add_rms_norm_backward, locals())
    lib = library()
    if not isinstance(h, _Tensor) or h.dim() < 1:
        raise ValueError("h must be a tensor [.., K]")
    shape = h.shape
    K = shape[-1]
    _need(h, "h", _FLOATS, shape)
    _need(g, "g", _FLOATS, shape)
    _opt(g_h, "g_h", h.dtype, shape)
    _opt(w, "w", torch.float32, (K,))
    if x_dtype is not None and x_dtype != h.dtype \
            and (x_dtype != torch.bfloat16 or h.dtype != torch.float32):
        raise ValueError("x_dtype must be h's type, or bfloat16 beside a float32 h")
    copy = x_dtype is not None and x_dtype != h.dtype
    _opt(dh, "dh", h.dtype, shape)
    if dx is not None and not copy:
        raise ValueError("dx is dh unless x_dtype differs from h's type")
    _opt(dx, "dx", torch.bfloat16, shape)
    if w is None and dw is not None:
        raise ValueError("dw given without w")
    _opt(dw, "dw", torch.float32, (K,))
    M = h.numel() // K if K else 0
    wsb = lib.convrot_add_rms_norm_workspace_bytes(M, K) if w is not None else 0
    _check_workspace(wsb, workspace)
    dev = _gpu_of(h)
    _on_device(dev, h=h, g=g, g_h=g_h, w=w, dh=dh, dx=dx, dw=dw, workspace=workspace)
    if dh is None:
        dh = torch.empty_like(h)
    if copy and dx is None:
        dx = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if w is not None and dw is None:
        dw = torch.empty(K, dtype=torch.float32, device=dev)
    ws = _workspace(wsb, dev, workspace)
    _launch(dev, "convrot_add_rms_norm_backward", _ptr(g), _dtype_tag(g.dtype), _ptr(h),
            _dtype_tag(h.dtype), _ptr(g_h), _ptr(w), eps, M, K, _ptr(dh), _ptr(dx), _ptr(dw),
            _ptr(ws), ws.numel() if ws is not None else 0)
    return dh, dx if copy else dh, dw


# ------------------------------------- mixture of experts for a few tokens ----

class MoEWeights:
    """The prepared experts of a layer: the C descriptor plus the tensors it points into."""

    def __init__(self, desc: convrot_moe_weights, gate_up, gate_up_scale, down, down_scale):
        self.desc = desc
        self.gate_up, self.gate_up_scale = gate_up, gate_up_scale
        self.down, self.down_scale = down, down_scale
        self._ref = ctypes.byref(desc)
        self._workspace = {}              # bytes by (tokens of a pass, top_k)

    @property
    def experts(self):
        return self.desc.experts

    @property
    def shared(self):
        return self.desc.shared

    @property
    def K(self):
        return self.desc.K

    @property
    def F(self):
        return self.desc.F

    def ref(self):
        return self._ref


def convrot_moe_prepare_weights(W_gate_up: torch.Tensor, W_down: torch.Tensor, shared: int = 0,
                                src_scale_gate_up=None, src_scale_down=None,
                                scales: str = "f32", stream=None) -> MoEWeights:
    """Pack the experts W_gate_up [E + S, 2F, K] (gate rows first) and W_down [E + S, K, F],
    the last S = shared of which serve every token: float32 or bfloat16, quantised to e4m3
    with a scale per 128 x 128 block, or float8_e4m3fn codes with their scales
    [E + S, 2F/128, K/128] and [E + S, K/128, F/128]."""
    if stream is not None:
        return _on_stream(convrot_moe_prepare_weights, locals())
    lib = library()
    for t, n in ((W_gate_up, "W_gate_up"), (W_down, "W_down")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{n} must be a 3-D tensor")
    n, K, F = W_down.shape
    dt = W_down.dtype
    if dt not in (torch.float32, torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"weights must be float32, bfloat16 or float8_e4m3fn codes, got {dt}")
    if W_gate_up.dtype != dt or tuple(W_gate_up.shape) != (n, 2 * F, K):
        raise ValueError(f"W_gate_up must be {dt} of shape {(n, 2 * F, K)}, got "
                         f"{W_gate_up.dtype} {tuple(W_gate_up.shape)}")
    if not 0 <= shared < max(n, 1):
        raise ValueError(f"shared must be from 0 to {max(n, 1) - 1}, got {shared}")
    if scales not in FP8_SCALES:
        raise ValueError(f"scales must be one of {sorted(FP8_SCALES)}")
    for t, rc, name in ((src_scale_gate_up, (2 * F, K), "src_scale_gate_up"),
                        (src_scale_down, (K, F), "src_scale_down")):
        if (dt == torch.float8_e4m3fn) != (t is not None):
            raise ValueError(f"{name} is required for float8_e4m3fn codes and only for them")
        _opt(t, name, torch.float32, (n, rc[0] // 128, rc[1] // 128))
    gub, db = lib.convrot_moe_packed_bytes(n, 2 * F, K), lib.convrot_moe_packed_bytes(n, K, F)
    if gub == 0 or db == 0:
        raise ConvRotError("convrot_moe_prepare_weights", EUNSUPPORTED)
    dev = W_down.device
    _on_device(None, W_down=W_down)
    _on_device(dev, W_gate_up=W_gate_up, src_scale_gate_up=src_scale_gate_up,
               src_scale_down=src_scale_down)
    W_gate_up, W_down = W_gate_up.contiguous(), W_down.contiguous()
    gate_up = torch.empty(gub, dtype=torch.uint8, device=dev)
    down = torch.empty(db, dtype=torch.uint8, device=dev)
    gus = torch.empty((n, 2 * F // 128, K // 128), dtype=torch.float32, device=dev)
    ds = torch.empty((n, K // 128, F // 128), dtype=torch.float32, device=dev)
    desc = convrot_moe_weights()
    desc.experts, desc.shared, desc.K, desc.F = n - shared, shared, K, F
    desc.gate_up, desc.gate_up_scale = gate_up.data_ptr(), gus.data_ptr()
    desc.down, desc.down_scale = down.data_ptr(), ds.data_ptr()
    _launch(dev, "convrot_moe_prepare_weights", _ptr(W_gate_up), _ptr(W_down), _dtype_tag(dt),
            _ptr(src_scale_gate_up), _ptr(src_scale_down), FP8_SCALES[scales],
            ctypes.byref(desc))
    return MoEWeights(desc, gate_up, gus, down, ds)


def convrot_moe_workspace_bytes(T: int, W: MoEWeights, top_k: int) -> int:
    return library().convrot_moe_workspace_bytes(T, W.ref(), top_k)


def convrot_moe_forward(X: torch.Tensor, router: torch.Tensor, W: MoEWeights, top_k: int,
                        router_bias=None, score: str = "softmax", renormalize: bool = True,
                        scale: float = 1.0, out_dtype: torch.dtype = torch.bfloat16, out=None,
                        ids=None, weights=None, workspace=None, stream=None):
    """(Y, ids, weights): the layer's output [T, K] for the bf16 tokens X [T, K], the experts
    each token chose [T, top_k] (int32, the largest first) and their weights (float32).
    router [E, K] bf16 or float32; router_bias float32 [E] acts on the choice alone.  Experts
    that no token chose are not read; beyond 64 tokens they are read once for every 64."""
    if stream is not None:
        return _on_stream(convrot_moe_forward, locals())
    if not isinstance(W, MoEWeights):
        raise ValueError("W must be MoEWeights from convrot_moe_prepare_weights")
    E, K = W.experts, W.K
    T = _rows(X, "X", K)
    _need(router, "router", _FLOATS, (E, K))
    _opt(router_bias, "router_bias", torch.float32, (E,))
    if score not in MOE_SCORES:
        raise ValueError(f"score must be one of {sorted(MOE_SCORES)}")
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k must be from 1 to {E}, got {top_k}")
    _opt(out, "out", _FLOATS, (T, K))
    _opt(ids, "ids", torch.int32, (T, top_k))
    _opt(weights, "weights", torch.float32, (T, top_k))
    key = min(T, MOE_PASS), top_k
    wsb = W._workspace.get(key)
    if wsb is None:
        wsb = W._workspace[key] = convrot_moe_workspace_bytes(T, W, top_k)
    _check_workspace(wsb, workspace)
    dev = W.down.device
    _on_device(dev, X=X, router=router, router_bias=router_bias, out=out, ids=ids,
               weights=weights, workspace=workspace)
    if out is None:
        out = _new(X, out_dtype)
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    ws = _workspace(wsb, dev, workspace)
    _launch(dev, "convrot_moe_forward", _ptr(X), T, _ptr(router), _dtype_tag(router.dtype),
            _ptr(router_bias), W.ref(), top_k, MOE_SCORES[score],
            MOE_RENORMALIZE if renormalize else 0, scale, _ptr(out), _dtype_tag(out.dtype),
            _ptr(ids), _ptr(weights), _ptr(ws), ws.numel() if ws is not None else 0)
    return out, ids, weights


# ------------------------------------------------------------- hooks ----

def padded_rows(M: int) -> int:
    """Rows of a K-tiled INT8 code buffer holding M rows (a multiple of 16)."""
    return (M + 15) // 16 * 16


def _codes(q, M: int, K: int, device):
    """A K-tiled code buffer for M rows of K codes: allocated as (Mp, K) int8
    on `device` when q is None, or a caller tensor checked to hold Mp * K
    bytes (its device is checked by the caller)."""
    Mp = padded_rows(M)
    if q is None:
        return torch.empty((Mp, K), dtype=torch.int8, device=device)
    if not isinstance(q, torch.Tensor) or q.dtype != torch.int8 or not q.is_contiguous() \
            or q.numel() < Mp * K:
        raise ValueError(f"K-tiled codes need a contiguous int8 tensor of {Mp * K} elements")
    return q


def convrot_rotate_quantize(X: torch.Tensor, block: int, q=None, s=None, stream=None,
                            rotation: str = "sylvester", gelu: bool = False):
    """Rotate + quantise the rows of X: (q, s), q the K-tiled codes (Mp, K).
    gelu: quantise bf16(GELU(X)) instead (bf16 X, 6144 < K <= 24576), as the
    MLP path does with its intermediate."""
    if stream is not None:
        return _on_stream(convrot_rotate_quantize, locals())
    lib = library()
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("X must be a 2-D tensor [M, K]")
    M, K = X.shape
    _need(X, "X", (torch.bfloat16, torch.float32), (M, K))
    q = _codes(q, M, K, X.device) if q is not None else None
    _opt(s, "s", torch.float32, (M,))
    if rotation not in ROTATIONS:
        raise ValueError(f"rotation must be one of {sorted(ROTATIONS)}")
    _on_device(X.device, X=X, q=q, s=s)
    if q is None:
        q = _codes(None, M, K, X.device)
    if s is None:
        s = torch.empty(M, dtype=torch.float32, device=X.device)
    flags = ROTATIONS[rotation] | (FLAG_GELU if gelu else 0)
    rc = lib.convrot_rotate_quantize(_ptr(X), _dtype_tag(X.dtype), M, K, block,
                                     flags, _ptr(q), _ptr(s), _stream(stream))
    _check("convrot_rotate_quantize", rc)
    return q, s


def convrot_gemm_i32(q_x: torch.Tensor, M: int, W: PreparedWeights, out=None, stream=None):
    """acc [M, N] int32 from K-tiled codes q_x of M rows."""
    if stream is not None:
        return _on_stream(convrot_gemm_i32, locals())
    lib = library()
    dev = _weights(W, "W")
    _codes(q_x, M, W.K, dev)
    _output(out, M, W.N, torch.int32)
    _on_device(dev, q_x=q_x, out=out)
    if out is None:
        out = torch.empty((M, W.N), dtype=torch.int32, device=dev)
    rc = lib.convrot_gemm_i32(_ptr(q_x), M, W.ref(), _ptr(out), _stream(stream))
    _check("convrot_gemm_i32", rc)
    return out


def convrot_gemm_dequant(q_x: torch.Tensor, s_x: torch.Tensor, W: PreparedWeights, bias=None,
                         out_dtype: torch.dtype = torch.bfloat16, out=None, gelu: bool = False,
                         swiglu: bool = False, stream=None):
    """Y [M, N] from K-tiled codes q_x and row scales s_x [M] (with swiglu, W a
    SwiGLU fc1 weight and Y = g [M, N/2])."""
    if stream is not None:
        return _on_stream(convrot_gemm_dequant, locals())
    lib = library()
    dev = _weights(W, "W")
    if not isinstance(s_x, torch.Tensor) or s_x.dim() != 1:
        raise ValueError("s_x must be a 1-D tensor [M]")
    M = s_x.shape[0]
    _need(s_x, "s_x", torch.float32, (M,))
    _codes(q_x, M, W.K, dev)
    _opt(bias, "bias", torch.float32, (W.N,))
    ncols = W.N // 2 if swiglu else W.N
    _output(out, M, ncols, (torch.bfloat16, torch.float32))
    _on_device(dev, q_x=q_x, s_x=s_x, bias=bias, out=out)
    if out is None:
        out = torch.empty((M, ncols), dtype=out_dtype, device=dev)
    flags = (FLAG_GELU if gelu else 0) | (FLAG_SWIGLU if swiglu else 0)
    rc = lib.convrot_gemm_dequant(_ptr(q_x), _ptr(s_x), M, W.ref(), _ptr(bias), _ptr(out),
                                  _dtype_tag(out.dtype), flags, _stream(stream))
    _check("convrot_gemm_dequant", rc)
    return out


def convrot_lowrank_factor1(q_x: torch.Tensor, s_x: torch.Tensor, A: PreparedWeights,
                            q_h=None, s_h=None, stream=None):
    """Factor 1 of the low-rank chain with its output rotated and requantised:
    returns (q_h, s_h), q_h the K-tiled codes (Mp, r), s_h [M] f32."""
    if stream is not None:
        return _on_stream(convrot_lowrank_factor1, locals())
    lib = library()
    dev = _weights(A, "A")
    if not isinstance(s_x, torch.Tensor) or s_x.dim() != 1:
        raise ValueError("s_x must be a 1-D tensor [M]")
    M = s_x.shape[0]
    _need(s_x, "s_x", torch.float32, (M,))
    _codes(q_x, M, A.K, dev)
    if q_h is not None:
        _codes(q_h, M, A.N, dev)
    _opt(s_h, "s_h", torch.float32, (M,))
    _on_device(dev, q_x=q_x, s_x=s_x, q_h=q_h, s_h=s_h)
    q_h = _codes(q_h, M, A.N, dev)
    if s_h is None:
        s_h = torch.empty(M, dtype=torch.float32, device=dev)
    rc = lib.convrot_lowrank_factor1(_ptr(q_x), _ptr(s_x), M, A.ref(), _ptr(q_h), _ptr(s_h),
                                     _stream(stream))
    _check("convrot_lowrank_factor1", rc)
    return q_h, s_h


def convrot_gelu_bf16(u: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """bf16(GELU(u)) elementwise, as the MLP's up projection applies it."""
    if stream is not None:
        return _on_stream(convrot_gelu_bf16, locals())
    lib = library()
    if not isinstance(u, torch.Tensor) or u.dtype != torch.bfloat16:
        raise ValueError("u must be a bf16 tensor")
    u = u.contiguous()
    _opt(out, "out", torch.bfloat16, tuple(u.shape))
    _on_device(u.device, u=u, out=out)
    if out is None:
        out = torch.empty_like(u)
    _check("convrot_gelu_bf16", lib.convrot_gelu_bf16(_ptr(u), u.numel(), _ptr(out),
                                                      _stream(stream)))
    return out


def convrot_fp8_quantize(X: torch.Tensor, scales: str = "f32", q=None, s=None, stream=None):
    """(q, s): the K-tiled e4m3 codes (Mp, K) uint8 of the bf16 rows X and their
    scales [K/128, Mp] float32."""
    if stream is not None:
        return _on_stream(convrot_fp8_quantize, locals())
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("X must be a 2-D tensor [M, K]")
    M, K = X.shape
    _need(X, "X", torch.bfloat16, (M, K))
    if scales not in FP8_SCALES:
        raise ValueError(f"scales must be one of {sorted(FP8_SCALES)}")
    Mp = padded_rows(M)
    _opt(q, "q", torch.uint8, (Mp, K))
    _opt(s, "s", torch.float32, (K // 128, Mp))
    _on_device(X.device, X=X, q=q, s=s)
    if q is None:
        q = torch.empty((Mp, K), dtype=torch.uint8, device=X.device)
    if s is None:
        s = torch.empty((K // 128, Mp), dtype=torch.float32, device=X.device)
    _launch(X.device, "convrot_fp8_quantize", _ptr(X), M, K, FP8_SCALES[scales], _ptr(q),
            _ptr(s))
    return q, s


def convrot_fp8_gemm_dequant(q: torch.Tensor, s: torch.Tensor, M: int, W: FP8Weights, bias=None,
                             out_dtype: torch.dtype = torch.bfloat16, out=None, stream=None,
                             scales: str = "f32"):
    """Y [M, N] from the codes and scales of M rows (convrot_fp8_quantize), of
    either kind.  scales='pow2' says that the rows' are powers of two or zeros
    (not checked): with a 'pow2' weight that is its forward's arithmetic."""
    if stream is not None:
        return _on_stream(convrot_fp8_gemm_dequant, locals())
    dev = _fp8_weights(W, "W")
    if scales not in FP8_SCALES:
        raise ValueError(f"scales must be one of {sorted(FP8_SCALES)}")
    _need(q, "q", torch.uint8, (padded_rows(M), W.K))
    _need(s, "s", torch.float32, (W.K // 128, padded_rows(M)))
    _opt(bias, "bias", torch.float32, (W.N,))
    _output(out, M, W.N, (torch.bfloat16, torch.float32))
    _on_device(dev, q=q, s=s, bias=bias, out=out)
    if out is None:
        out = torch.empty((M, W.N), dtype=out_dtype, device=dev)
    _launch(dev, "convrot_fp8_gemm_dequant_scales", _ptr(q), _ptr(s), FP8_SCALES[scales],
            M, W.ref(), _ptr(bias), _ptr(out), _dtype_tag(out.dtype))
    return out


def convrot_probe_mfma_i8(iters: int, seed: torch.Tensor, sink: torch.Tensor,
                          stream=None) -> int:
    """Launch the INT8 MFMA rate probe; returns its INT8 operation count.
    seed: 4 KiB on the device (the operands it starts from); sink: 16 bytes."""
    lib = library()
    if seed.numel() * seed.element_size() < 4096 or sink.numel() * sink.element_size() < 16:
        raise ValueError("seed needs 4 KiB and sink 16 bytes")
    ops = ctypes.c_int64(0)
    _check("convrot_probe_mfma_i8", lib.convrot_probe_mfma_i8(
        iters, _ptr(seed), _ptr(sink), ctypes.byref(ops), _stream(stream)))
    return ops.value


def convrot_probe_stream(src, dst: torch.Tensor, mode: int, stream=None):
    """Streaming probe: mode 0 reads src's 16-byte items and writes 8 bytes
    per item into dst, mode 1 copies them, mode 2 (src None) only writes all
    of dst's 16-byte items."""
    lib = library()
    if mode == 2:
        n16 = dst.numel() * dst.element_size() // 16
    else:
        nbytes = src.numel() * src.element_size()
        n16 = nbytes // 16
        if nbytes % 16 or dst.numel() * dst.element_size() < n16 * (8 if mode == 0 else 16):
            raise ValueError("src must be whole 16-byte items and dst large enough")
    _check("convrot_probe_stream", lib.convrot_probe_stream(
        None if src is None else _ptr(src), _ptr(dst), n16, mode, _stream(stream)))
    return dst
