"""Python binding of libfp8_moe_grouped.so, the MI355X (gfx950) routed-expert
FP8 grouped-matmul library.

Argument marshalling only: each function checks dtypes, shapes, devices and
contiguity of torch tensors, allocates outputs and the device workspace with
torch (torch is used for device memory and streams), and calls the C entry
point of the same name on the current HIP stream.  Every step of the
computation runs in the library's HIP kernels; there is no fallback.  If the
shared library is missing the first call raises.

The calls around the products (routing, balance losses, dispatch, combine, weight
quantizers, AdamW, 4-bit) first hand their arguments to a small extension (csrc/calls.cpp), which makes the same C
call without the interpreter's checks where the arguments are the plain ones;
it answers None otherwise, and the function here checks, calls and reports.

The C contract of every call is documented in include/fp8_moe_grouped.h.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
import re
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8_moe_grouped.so")
CALLS_PATH = os.path.join(_HERE, "_calls.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "fp8_moe_grouped.h")

OK = 0
ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE, ERR_HIP, ERR_SCRATCH = -1, -2, -3, -4, -5, -6, -7
ERR_OVERLAP = -8
NOALLOC_SCRATCH_BYTES = 32 << 20
DEV_SUM_CLAMPED, DEV_NEGATIVE_SIZE = 1, 2
E4M3, E5M2 = 0, 1
(OP_FWD, OP_SILU, OP_DLHS, OP_TGMM, OP_BF16_FWD, OP_BF16_DLHS, OP_FFN_FWD, OP_FFN_BWD, OP_FWD_VARIANT,
 OP_TGMM_DENSE, OP_ROUTE, OP_MXFP4, OP_BALANCE, OP_QUANT_WEIGHTS) = range(14)
LHS_SCALE_BF16, ACC_BF16, RHS_SCALE_FIRST = 1, 2, 4
GRAD_DTYPES = {"e4m3": E4M3, "e5m2": E5M2}
F32, BF16 = 0, 1
LOGIT_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class Fp8GmmError(RuntimeError):
    """A library call returned a non-zero status."""

    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__(f"{call}: {status_string(status)} (status {status})")


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_U64 = ctypes.c_uint64
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "gmm_fp8_fwd": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "gmm_fp8_fwd_noalloc": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P],
    "gmm_silu_fp8": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _P, _SZ, _P, _P],
    "gmm_dlhs_fp8": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _SZ, _P, _P],
    "tgmm_quant": [_P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "dequantize_fp8_codes": [_P, _P, _I32, _I64, _I64, _P, _P],
    "tgmm_dense_quant": [_P, _P, _P, _I64, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "quantize_rows_fp8": [_P, _P, _I64, _I64, _I32, _P, _P, _P],
    "gmm_fp8_fwd_q": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P],
    "gmm_silu_fp8_q": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P, _P],
    "gmm_fp8_fwd_variant": [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "gmm_dswiglu_fp8": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P],
    "moe_ffn_fp8_fwd": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "moe_ffn_fp8_bwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P,
                        _SZ, _P, _P],
    "gmm_bf16_fwd": [_P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P],
    "gmm_bf16_silu": [_P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P],
    "gmm_bf16_dlhs": [_P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P],
    "moe_route": [_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "moe_route_bwd": [_P, _P, _I32, _P, _P, _I64, _I32, _I32, _I32, _P, _P],
    "moe_permute": [_P, _P, _I64, _I32, _I64, _I64, _P, _P],
    "moe_permute_fp8": [_P, _P, _I64, _I32, _I64, _I64, _P, _P, _P],
    "moe_combine": [_P, _P, _P, _I64, _I32, _I64, _I64, _P, _P],
    "moe_combine_bwd": [_P, _P, _P, _P, _I64, _I32, _I64, _I64, _P, _P, _P],
    "moe_balance_loss": [_P, _I32, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P],
    "moe_balance_loss_bwd": [_P, _P, _I32, _P, _P, _I64, _I32, _P, _P, _P],
    "adamw_step": [_I32, _P, _P, _I32, _P, _I32, _P, _P, _P, _P],
    "adamw_step_8bit": [_I32, _P, _P, _I32, _P, _I32, _P, _P, _P, _P, _U64, _P, _P],
    "quantize_fp8_weights": [_P, _I32, _I64, _I64, _I32, _P, _P, _P, _SZ, _P],
    "quantize_mxfp4_weights": [_P, _I64, _I64, _I32, _P, _P, _P],
    "dequantize_mxfp4": [_P, _P, _I64, _I64, _I32, _P, _P],
    "gmm_mxfp4_fwd": [_P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I64, _I32, _P, _P, _SZ, _P, _P],
    "gmm_silu_mxfp4": [_P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I64, _I32, _P, _P, _SZ, _P, _P],
}

_lib = None
_calls = None


def _plain():
    """The extension of csrc/calls.cpp on the library's entry points."""
    global _calls
    if _calls is None:
        L = lib()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} is missing: build it first (python -m fp8_moe_grouped_amd.build)")
        spec = importlib.util.spec_from_file_location("fp8_moe_grouped_amd._calls", CALLS_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.bind(*(ctypes.cast(getattr(L, name), _P).value for name in m.names()))
        _calls = m
    return _calls


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -m fp8_moe_grouped_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.fp8gmm_workspace_bytes.argtypes = [_I32, _I64, _I64, _I64, _I32, _I32]
        L.fp8gmm_workspace_bytes.restype = ctypes.c_size_t
        L.fp8gmm_status_string.argtypes = [_I32]
        L.fp8gmm_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/fp8_moe_grouped.h."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:int|size_t|const char\s*\*)\s*(\w+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    return lib().fp8gmm_status_string(int(status)).decode()


def workspace_bytes(op: int, M: int, K: int, N: int, G: int, tile_m: int = 512) -> int:
    return int(lib().fp8gmm_workspace_bytes(op, M, K, N, G, tile_m))


# --------------------------------------------------------------------------- marshalling

# What a call costs the host counts beside kernels of a few microseconds: plain
# integers for pointers, the current stream's handle without a Stream object
# (0.1 us, not 2), and no device switch where the device is the current one
# already (0.2 us, not 1.4).

def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


_HERE_ALREADY = contextlib.nullcontext()


def _on(dev):
    """A context in which dev is the current device."""
    return _HERE_ALREADY if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _req(t, name, dtype, ndim):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.dim() == ndim and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _req_i32(v, name):
    """ctypes would keep the low 32 bits."""
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {v}")


def _same_device(*ts):
    dev = None
    for t in ts:
        if not isinstance(t, torch.Tensor):         # None, or refused by its own check
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"all tensors must be on one device, got {set(t.device for t in ts if t is not None)}")
    return dev


def _call(name, *args):
    st = getattr(lib(), name)(*args)
    if st != OK:
        raise Fp8GmmError(name, st)


def _launch(dev, name, *args):
    """Calls entry point `name` on dev's current stream (its last argument)."""
    fn = getattr(_lib or lib(), name)
    if torch._C._cuda_getDevice() == dev.index:
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st != OK:
        raise Fp8GmmError(name, st)


def _workspace(op, M, K, N, G, dev, tile_m=512, workspace=None):
    need = workspace_bytes(op, M, K, N, G, tile_m)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.numel() < need:
        raise ValueError(f"workspace has {workspace.numel()} bytes, {need} needed")
    return workspace, need


def _fwd(name, op, lhs, codes, scale, group_sizes, out, debug, dev_status, workspace, swiglu, preact=None):
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, codes, scale, group_sizes)
    M, K = lhs.shape
    G, K2, N = codes.shape
    if K2 != K or tuple(scale.shape) != (G, N) or group_sizes.shape[0] != G:
        raise ValueError(f"shape mismatch: lhs {tuple(lhs.shape)} codes {tuple(codes.shape)} "
                         f"scale {tuple(scale.shape)} group_sizes {tuple(group_sizes.shape)}")
    ncol = N // 2 if swiglu else N
    if out is None:
        out = torch.empty((M, ncol), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, 2)
    if preact is True:
        preact = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if preact is not None:
        _req(preact, "preact", torch.bfloat16, 2)
        if tuple(preact.shape) != (M, N):
            raise ValueError(f"preact must be [{M}, {N}], got {tuple(preact.shape)}")
    dbg_codes = torch.empty((M, K), dtype=torch.uint8, device=dev) if debug else None
    dbg_scale = torch.empty((M,), dtype=torch.float32, device=dev) if debug else None
    ws, need = _workspace(op, M, K, N, G, dev, workspace=workspace)
    extra = (_ptr(preact),) if swiglu else ()
    with _on(dev):
        _call(name, _ptr(lhs), _ptr(codes), _ptr(scale), _ptr(group_sizes), M, K, N, G, _ptr(out), *extra,
              _ptr(dbg_codes), _ptr(dbg_scale), _ptr(ws), need, _ptr(dev_status), _stream(dev))
    res = (out,) + ((preact,) if preact is not None else ()) + ((dbg_codes, dbg_scale) if debug else ())
    return res if len(res) > 1 else out


def gmm_fp8_fwd(lhs, codes, scale, group_sizes, *, out=None, debug=False, dev_status=None, workspace=None):
    """Native FP8 forward GMM; returns bf16 [M, N] (and, with debug, the
    activation codes [M, K] and row scales [M] the GEMM consumed)."""
    return _fwd("gmm_fp8_fwd", OP_FWD, lhs, codes, scale, group_sizes, out, debug, dev_status, workspace, False)


def gmm_fp8_fwd_noalloc(lhs, codes, scale, group_sizes, *, out=None, dev_status=None):
    """gmm_fp8_fwd through the allocation-free entry point: the library keeps
    the quantized activations in its fixed per-GPU scratch (the call itself
    allocates nothing; only ``out``, if not given, is allocated here).
    Returns bf16 [M, N]."""
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, codes, scale, group_sizes)
    M, K = lhs.shape
    G, K2, N = codes.shape
    if K2 != K or tuple(scale.shape) != (G, N) or group_sizes.shape[0] != G:
        raise ValueError("shape mismatch")
    out = _out(out, (M, N), torch.bfloat16, dev, "out")
    with _on(dev):
        _call("gmm_fp8_fwd_noalloc", _ptr(lhs), _ptr(codes), _ptr(scale), _ptr(group_sizes), M, K, N, G, _ptr(out),
              _ptr(dev_status), _stream(dev))
    return out


def gmm_silu_fp8(lhs, codes, scale, group_sizes, *, out=None, preact=None, debug=False, dev_status=None,
                 workspace=None):
    """Native FP8 forward GMM with fused SwiGLU over [gate | up]; bf16 [M, N/2].
    ``preact`` (a bf16 [M, N] tensor, or True to allocate one) also receives
    the pre-activation; the result is then ``(out, preact)`` (followed by the
    debug outputs when asked)."""
    return _fwd("gmm_silu_fp8", OP_SILU, lhs, codes, scale, group_sizes, out, debug, dev_status, workspace, True,
                preact)


def gmm_fp8_fwd_variant(lhs, codes, scale, group_sizes, *, lhs_block=0, scale_bf16=False, acc_bf16=False,
                        rhs_scale_first=False, out=None, debug=False, dev_status=None, workspace=None):
    """The FP8 forward with the ops-level LHS-quantization options: one scale
    per row (lhs_block=0) or per 512 columns, optionally rounded to bf16, a
    bf16 accumulator across the 512-column blocks, and the weight scale
    applied first.  Returns bf16 [M, N] (with debug also the codes [M, K] and
    the scales [M, nb])."""
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, codes, scale, group_sizes)
    M, K = lhs.shape
    G, K2, N = codes.shape
    if K2 != K or tuple(scale.shape) != (G, N) or group_sizes.shape[0] != G:
        raise ValueError("shape mismatch")
    flags = (LHS_SCALE_BF16 if scale_bf16 else 0) | (ACC_BF16 if acc_bf16 else 0) | \
        (RHS_SCALE_FIRST if rhs_scale_first else 0)
    nb = -(-K // 512) if lhs_block == 512 else 1
    out = _out(out, (M, N), torch.bfloat16, dev, "out")
    dbg_codes = torch.empty((M, K), dtype=torch.uint8, device=dev) if debug else None
    dbg_scale = torch.empty((M, nb), dtype=torch.float32, device=dev) if debug else None
    ws, need = _workspace(OP_FWD_VARIANT, M, K, N, G, dev, tile_m=lhs_block, workspace=workspace)
    with _on(dev):
        _call("gmm_fp8_fwd_variant", _ptr(lhs), _ptr(codes), _ptr(scale), _ptr(group_sizes), M, K, N, G,
              int(lhs_block), flags, _ptr(out), _ptr(dbg_codes), _ptr(dbg_scale), _ptr(ws), need, _ptr(dev_status),
              _stream(dev))
    return (out, dbg_codes, dbg_scale) if debug else out


def quantize_rows_fp8(lhs, group_sizes, *, codes=None, scales=None):
    """e4m3 codes [M, K] and f32 row scales [M] of the valid rows (the first
    half of gmm_fp8_fwd); rows past the valid prefix are left untouched."""
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, group_sizes)
    M, K = lhs.shape
    if codes is None:
        codes = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((M,), dtype=torch.float32, device=dev)
    _req(codes, "codes", torch.uint8, 2)
    _req(scales, "scales", torch.float32, 1)
    with _on(dev):
        _call("quantize_rows_fp8", _ptr(lhs), _ptr(group_sizes), M, K, group_sizes.shape[0], _ptr(codes),
              _ptr(scales), _stream(dev))
    return codes, scales


def _fwd_q(name, aq, ascale, codes, scale, group_sizes, out, dev_status, swiglu, preact=None):
    _req(aq, "aq", torch.uint8, 2)
    _req(ascale, "ascale", torch.float32, 1)
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(aq, ascale, codes, scale, group_sizes)
    M, K = aq.shape
    G, K2, N = codes.shape
    if K2 != K or tuple(scale.shape) != (G, N) or group_sizes.shape[0] != G or ascale.shape[0] != M:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, N // 2 if swiglu else N), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, 2)
    if preact is not None:
        _req(preact, "preact", torch.bfloat16, 2)
        if tuple(preact.shape) != (M, N):
            raise ValueError(f"preact must be [{M}, {N}], got {tuple(preact.shape)}")
    extra = (_ptr(preact),) if swiglu else ()
    with _on(dev):
        _call(name, _ptr(aq), _ptr(ascale), _ptr(codes), _ptr(scale), _ptr(group_sizes), M, K, N, G, _ptr(out),
              *extra, _ptr(dev_status), _stream(dev))
    return out


def gmm_fp8_fwd_q(aq, ascale, codes, scale, group_sizes, *, out=None, dev_status=None):
    """FP8 forward GEMM on already quantized activations (codes + row scales)."""
    return _fwd_q("gmm_fp8_fwd_q", aq, ascale, codes, scale, group_sizes, out, dev_status, False)


def gmm_silu_fp8_q(aq, ascale, codes, scale, group_sizes, *, out=None, preact=None, dev_status=None):
    """FP8 forward GEMM + SwiGLU on already quantized activations; a bf16
    [M, N] ``preact`` tensor, if given, receives the pre-activation."""
    return _fwd_q("gmm_silu_fp8_q", aq, ascale, codes, scale, group_sizes, out, dev_status, True, preact)


def gmm_dlhs_fp8(dout, codes, scale, group_sizes, *, out=None, dev_status=None, workspace=None):
    """Backward dLHS from FP8 codes; returns bf16 [M, K]."""
    _req(dout, "dout", torch.bfloat16, 2)
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(dout, codes, scale, group_sizes)
    M, N = dout.shape
    G, K, N2 = codes.shape
    if N2 != N or tuple(scale.shape) != (G, N) or group_sizes.shape[0] != G:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, 2)
    ws, need = _workspace(OP_DLHS, M, K, N, G, dev, workspace=workspace)
    with _on(dev):
        _call("gmm_dlhs_fp8", _ptr(dout), _ptr(codes), _ptr(scale), _ptr(group_sizes), M, K, N, G, _ptr(out),
              _ptr(ws), need, _ptr(dev_status), _stream(dev))
    return out


def gmm_dswiglu_fp8(dout, codes, scale, group_sizes, preact, *, out=None, dev_status=None):
    """wo backward dLHS fused with the SwiGLU derivative: from the wo output
    gradient dout [M, H], the wo codes [G, I, H] and the wi pre-activation
    preact [M, 2I], returns the pre-activation gradient bf16 [M, 2I]."""
    _req(dout, "dout", torch.bfloat16, 2)
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    _req(preact, "preact", torch.bfloat16, 2)
    dev = _same_device(dout, codes, scale, group_sizes, preact)
    M, N = dout.shape
    G, K, N2 = codes.shape
    if N2 != N or tuple(scale.shape) != (G, N) or group_sizes.shape[0] != G or tuple(preact.shape) != (M, 2 * K):
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, 2 * K), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, 2 * K):
        raise ValueError("out must be [M, 2K]")
    with _on(dev):
        _call("gmm_dswiglu_fp8", _ptr(dout), _ptr(codes), _ptr(scale), _ptr(group_sizes), _ptr(preact), M, K, N, G,
              _ptr(out), _ptr(dev_status), _stream(dev))
    return out


def _ffn_shapes(x, wi_codes, wi_scale, wo_codes, wo_scale, group_sizes):
    _req(x, "x", torch.bfloat16, 2)
    _req(wi_codes, "wi_codes", torch.uint8, 3)
    _req(wi_scale, "wi_scale", torch.float32, 2)
    _req(wo_codes, "wo_codes", torch.uint8, 3)
    _req(wo_scale, "wo_scale", torch.float32, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(x, wi_codes, wi_scale, wo_codes, wo_scale, group_sizes)
    M, H = x.shape
    G, H2, I2 = wi_codes.shape
    I = I2 // 2
    if (H2 != H or I2 != 2 * I or tuple(wi_scale.shape) != (G, I2) or tuple(wo_codes.shape) != (G, I, H)
            or tuple(wo_scale.shape) != (G, H) or group_sizes.shape[0] != G):
        raise ValueError(f"FFN shape mismatch: x {tuple(x.shape)} wi {tuple(wi_codes.shape)} "
                         f"wo {tuple(wo_codes.shape)}")
    return dev, M, H, I, G


def _out(t, shape, dtype, dev, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _req(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def moe_ffn_fp8_fwd(x, wi_codes, wi_scale, wo_codes, wo_scale, group_sizes, *, keep_preact=True, h=None,
                    preact=None, y=None, dev_status=None, workspace=None):
    """Forward of one routed-expert FFN: h = SwiGLU FP8 GMM of x with wi,
    y = FP8 GMM of h with wo.  Returns (y [M, H], h [M, I], preact [M, 2I] or
    None)."""
    dev, M, H, I, G = _ffn_shapes(x, wi_codes, wi_scale, wo_codes, wo_scale, group_sizes)
    h = _out(h, (M, I), torch.bfloat16, dev, "h")
    y = _out(y, (M, H), torch.bfloat16, dev, "y")
    preact = _out(preact, (M, 2 * I), torch.bfloat16, dev, "preact") if (keep_preact or preact is not None) else None
    ws, need = _workspace(OP_FFN_FWD, M, H, I, G, dev, tile_m=0, workspace=workspace)
    with _on(dev):
        _call("moe_ffn_fp8_fwd", _ptr(x), _ptr(wi_codes), _ptr(wi_scale), _ptr(wo_codes), _ptr(wo_scale),
              _ptr(group_sizes), M, H, I, G, _ptr(h), _ptr(preact), _ptr(y), _ptr(ws), need, _ptr(dev_status),
              _stream(dev))
    return y, h, preact


def moe_ffn_fp8_bwd(x, h, preact, dy, wi_codes, wi_scale, wo_codes, wo_scale, group_sizes, grad_dtype="e5m2", *,
                    need_dx=True, d_preact=None, dx=None, dwi=None, dwo=None, dev_status=None, workspace=None):
    """Backward of one routed-expert FFN from the forward's x, h, preact and
    the output gradient dy [M, H].  Returns (dx [M, H] or None, dwi
    [G, H, 2I] f32, dwo [G, I, H] f32, d_preact [M, 2I])."""
    dev, M, H, I, G = _ffn_shapes(x, wi_codes, wi_scale, wo_codes, wo_scale, group_sizes)
    for t, name, shape in ((h, "h", (M, I)), (preact, "preact", (M, 2 * I)), (dy, "dy", (M, H))):
        _req(t, name, torch.bfloat16, 2)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    _same_device(x, h, preact, dy)
    gd = GRAD_DTYPES[grad_dtype] if isinstance(grad_dtype, str) else int(grad_dtype)
    d_preact = _out(d_preact, (M, 2 * I), torch.bfloat16, dev, "d_preact")
    dx = _out(dx, (M, H), torch.bfloat16, dev, "dx") if (need_dx or dx is not None) else None
    dwi = _out(dwi, (G, H, 2 * I), torch.float32, dev, "dwi")
    dwo = _out(dwo, (G, I, H), torch.float32, dev, "dwo")
    ws, need = _workspace(OP_FFN_BWD, M, H, I, G, dev, tile_m=512, workspace=workspace)
    with _on(dev):
        _call("moe_ffn_fp8_bwd", _ptr(x), _ptr(h), _ptr(preact), _ptr(dy), _ptr(wi_codes), _ptr(wi_scale),
              _ptr(wo_codes), _ptr(wo_scale), _ptr(group_sizes), M, H, I, G, gd, _ptr(d_preact), _ptr(dx),
              _ptr(dwi), _ptr(dwo), _ptr(ws), need, _ptr(dev_status), _stream(dev))
    return dx, dwi, dwo, d_preact


def tgmm_quant(lhs, dout, group_sizes, grad_dtype="e5m2", tile_m=512, *, out=None, debug=False,
               dev_status=None, workspace=None):
    """Weight-gradient tgmm with in-kernel per-(tile, channel) operand
    quantization; returns f32 [G, K, N] (and, with debug, the scales sL
    [Tmax, K] and sD [Tmax, N] of the non-empty (expert, tile) pairs)."""
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(dout, "dout", torch.bfloat16, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, dout, group_sizes)
    M, K = lhs.shape
    M2, N = dout.shape
    G = group_sizes.shape[0]
    if M2 != M:
        raise ValueError("lhs and dout must have the same number of rows")
    gd = GRAD_DTYPES[grad_dtype] if isinstance(grad_dtype, str) else int(grad_dtype)
    if out is None:
        out = torch.empty((G, K, N), dtype=torch.float32, device=dev)
    _req(out, "out", torch.float32, 3)
    tmax = -(-M // tile_m) + G - 1 if tile_m > 0 else 0
    dbg_sL = torch.empty((max(tmax, 1), K), dtype=torch.float32, device=dev) if debug else None
    dbg_sD = torch.empty((max(tmax, 1), N), dtype=torch.float32, device=dev) if debug else None
    ws, need = _workspace(OP_TGMM, M, K, N, G, dev, tile_m=tile_m, workspace=workspace)
    with _on(dev):
        _call("tgmm_quant", _ptr(lhs), _ptr(dout), _ptr(group_sizes), M, K, N, G, gd, tile_m, _ptr(out),
              _ptr(dbg_sL), _ptr(dbg_sD), _ptr(ws), need, _ptr(dev_status), _stream(dev))
    return (out, dbg_sL, dbg_sD) if debug else out


def tgmm_workspace_codes(workspace, M, K, N, G, tile_m=512):
    """Views of the operand codes a tgmm_quant call left in its workspace
    (the layout the header documents): qL uint8 [Tmax, tile_m, K] and qD
    uint8 [Tmax, tile_m, N], one slab per non-empty (expert, tile) pair in
    (expert, tile) order; slab p holds the pair's rows in order, then zero
    codes up to the next multiple of 32 rows."""
    tmax = -(-M // tile_m) + G - 1
    al = lambda x: (x + 255) // 256 * 256
    need = workspace_bytes(OP_TGMM, M, K, N, G, tile_m)
    if workspace.numel() < need or tmax <= 0:
        raise ValueError("workspace too small for these sizes")
    ql = workspace[: tmax * tile_m * K].view(tmax, tile_m, K)
    off = al(tmax * tile_m * K)
    qd = workspace[off: off + tmax * tile_m * N].view(tmax, tile_m, N)
    return ql, qd


def tgmm_workspace_deal(workspace, M, K, N, G, tile_m=512):
    """View of the GEMM's work-item deal a tgmm_quant call left in its
    workspace (the layout the header documents): int32 [G] block offsets."""
    tmax = -(-M // tile_m) + G - 1
    al = lambda x: (x + 255) // 256 * 256
    off = al(tmax * tile_m * K) + al(tmax * tile_m * N) + al(tmax * K * 4) + al(tmax * N * 4)
    if workspace.numel() < off + 4 * G or tmax <= 0:
        raise ValueError("workspace too small for these sizes")
    return workspace[off: off + 4 * G].view(torch.int32)


def tgmm_dense_quant(lhs, dout, group_sizes, grad_dtype="e5m2", *, out=None, debug=False, dev_status=None,
                     workspace=None):
    """The buffer-wide backward quantization baseline (every row of the
    buffer, stale rows included): per-row lhs scale folded into dout, one
    gradient scale per column; returns f32 [G, K, N] (with debug also the row
    scales [M] and the column scales [N])."""
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(dout, "dout", torch.bfloat16, 2)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, dout, group_sizes)
    M, K = lhs.shape
    M2, N = dout.shape
    G = group_sizes.shape[0]
    if M2 != M:
        raise ValueError("lhs and dout must have the same number of rows")
    gd = GRAD_DTYPES[grad_dtype] if isinstance(grad_dtype, str) else int(grad_dtype)
    out = _out(out, (G, K, N), torch.float32, dev, "out")
    srow = torch.empty((max(M, 1),), dtype=torch.float32, device=dev) if debug else None
    scol = torch.empty((N,), dtype=torch.float32, device=dev) if debug else None
    ws, need = _workspace(OP_TGMM_DENSE, M, K, N, G, dev, tile_m=0, workspace=workspace)
    with _on(dev):
        _call("tgmm_dense_quant", _ptr(lhs), _ptr(dout), _ptr(group_sizes), M, K, N, G, gd, _ptr(out), _ptr(srow),
              _ptr(scol), _ptr(ws), need, _ptr(dev_status), _stream(dev))
    return (out, srow, scol) if debug else out


def dequantize_fp8_codes(codes, scale, *, out=None):
    """bf16 [G, K, N] = bf16(f32(dec(codes) * scale))."""
    _req(codes, "codes", torch.uint8, 3)
    _req(scale, "scale", torch.float32, 2)
    dev = _same_device(codes, scale)
    G, K, N = codes.shape
    if tuple(scale.shape) != (G, N):
        raise ValueError("scale must be [G, N]")
    if out is None:
        out = torch.empty((G, K, N), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, 3)
    with _on(dev):
        _call("dequantize_fp8_codes", _ptr(codes), _ptr(scale), G, K, N, _ptr(out), _stream(dev))
    return out


def _bf16_fwd(name, lhs, w, group_sizes, out, swiglu, dev_status):
    _req(lhs, "lhs", torch.bfloat16, 2)
    _req(w, "w", torch.bfloat16, 3)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(lhs, w, group_sizes)
    M, K = lhs.shape
    G, K2, N = w.shape
    if K2 != K or group_sizes.shape[0] != G:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, N // 2 if swiglu else N), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, 2)
    with _on(dev):
        _call(name, _ptr(lhs), _ptr(w), _ptr(group_sizes), M, K, N, G, _ptr(out), _ptr(dev_status), _stream(dev))
    return out


def gmm_bf16_fwd(lhs, w, group_sizes, *, out=None, dev_status=None):
    """bf16 x bf16 grouped GEMM (the bf16 measurement arm); bf16 [M, N]."""
    return _bf16_fwd("gmm_bf16_fwd", lhs, w, group_sizes, out, False, dev_status)


def gmm_bf16_silu(lhs, w, group_sizes, *, out=None, dev_status=None):
    """bf16 grouped GEMM with the SwiGLU epilogue over [gate | up] (the bf16
    arm of gmm_silu_fp8); bf16 [M, N/2]."""
    return _bf16_fwd("gmm_bf16_silu", lhs, w, group_sizes, out, True, dev_status)


def gmm_bf16_dlhs(dout, w, group_sizes, *, out=None):
    """bf16 dLHS with bf16 weights w [G, K, N] (the bf16 measurement arm and
    the bit-identity reference of gmm_dlhs_fp8); bf16 [M, K]."""
    _req(dout, "dout", torch.bfloat16, 2)
    _req(w, "w", torch.bfloat16, 3)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    dev = _same_device(dout, w, group_sizes)
    M, N = dout.shape
    G, K, N2 = w.shape
    if N2 != N or group_sizes.shape[0] != G:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    with _on(dev):
        _call("gmm_bf16_dlhs", _ptr(dout), _ptr(w), _ptr(group_sizes), M, K, N, G, _ptr(out), None, _stream(dev))
    return out


# --------------------------------------------------------------------------- routing, dispatch, combine

class MoeRouting(NamedTuple):
    """What moe_route returns; a slot is one of a token's k choices."""
    ids: torch.Tensor          # int32 [T, k], -1 for a choice that found only masked logits
    weights: torch.Tensor      # float32 [T, k]
    group_sizes: torch.Tensor  # int32 [E]
    row_of_slot: torch.Tensor  # int32 [T, k], -1 where ids is
    slot_of_row: torch.Tensor  # int32 [T * k], -1 past the last slot's row


def _req_logits(logits):
    if isinstance(logits, torch.Tensor) and logits.dtype not in LOGIT_DTYPES:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    _req(logits, "logits", getattr(logits, "dtype", None), 2)


def _req_slots(t, name, dtype, T, k):
    _req(t, name, dtype, 2)
    if t.shape != (T, k):
        raise ValueError(f"{name} must be [{T}, {k}], got {tuple(t.shape)}")


def moe_route(logits, k, *, renormalize=True, workspace=None):
    """The k largest of each token's router logits [T, E] (float32 or bfloat16;
    -inf masks an expert), their softmax weights (over the chosen experts, or
    over all without ``renormalize``) and the slots' stable sort by expert:
    a MoeRouting."""
    k = int(k)
    if workspace is None:
        r = (_calls or _plain()).route(logits, k, renormalize)
        if r is not None:
            return MoeRouting._make(r)
    _req_logits(logits)
    dev = logits.device
    T, E = logits.shape
    _req_i32(E, "the number of experts")
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, 1)
        _same_device(logits, workspace)
    if not 1 <= k <= E:
        raise ValueError(f"k must be between 1 and the {E} experts, got {k}")
    # one allocation for the four outputs of a slot (a view costs the host less than a tensor)
    ids, weights, row_of_slot, slot_of_row = torch.empty((4, T, k), dtype=torch.int32, device=dev).unbind(0)
    weights, slot_of_row = weights.view(torch.float32), slot_of_row.view(-1)
    group_sizes = torch.empty((E,), dtype=torch.int32, device=dev)
    ws, need = _workspace(OP_ROUTE, T, E, k, 1, dev, tile_m=0, workspace=workspace)
    _launch(dev, "moe_route", _ptr(logits), LOGIT_DTYPES[logits.dtype], T, E, k, bool(renormalize), _ptr(ids),
            _ptr(weights), _ptr(group_sizes), _ptr(row_of_slot), _ptr(slot_of_row), _ptr(ws), need)
    return MoeRouting(ids, weights, group_sizes, row_of_slot, slot_of_row)


def moe_route_bwd(dweights, logits, ids, weights, *, renormalize=True, out=None):
    """The gradient of moe_route's weights by its logits, in the logits' type
    [T, E], from dweights [T, k] and the call's logits, ids and weights."""
    if out is None:
        out = (_calls or _plain()).route_bwd(dweights, logits, ids, weights, renormalize)
        if out is not None:
            return out
    _req_logits(logits)
    T, E = logits.shape
    _req(ids, "ids", torch.int32, 2)
    k = ids.shape[1]
    _req_i32(max(E, k), "a side of logits and ids")
    if ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}, k], got {tuple(ids.shape)}")
    _req_slots(weights, "weights", torch.float32, T, k)
    _req_slots(dweights, "dweights", torch.float32, T, k)
    dev = _same_device(dweights, logits, ids, weights, out)
    out = _out(out, (T, E), logits.dtype, dev, "out")
    _launch(dev, "moe_route_bwd", _ptr(dweights), _ptr(logits), LOGIT_DTYPES[logits.dtype], _ptr(ids), _ptr(weights), T,
            E, k, bool(renormalize), _ptr(out))
    return out


def _slots(x, name, row_of_slot, rows, *others):
    """(device, T, k, H) of bf16 rows x and the map; `rows` if x has a row a
    token.  All tensors given are on the device."""
    _req(x, name, torch.bfloat16, 2)
    _req(row_of_slot, "row_of_slot", torch.int32, 2)
    T, k = row_of_slot.shape
    R, H = x.shape
    _req_i32(k, "k")
    if rows and R != T:
        raise ValueError(f"{name} must have the {T} rows of row_of_slot, got {tuple(x.shape)}")
    return _same_device(x, row_of_slot, *others), T, k, H


def moe_permute(x, row_of_slot, *, out=None):
    """bf16 [R, H]: row row_of_slot[t, j] is x[t] (R = T * k, or the rows of
    ``out``); rows that no slot names are left as they are."""
    if out is None:
        out = (_calls or _plain()).permute(x, row_of_slot)
        if out is not None:
            return out
    dev, T, k, H = _slots(x, "x", row_of_slot, True, out)
    if out is None:
        out = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev)
    else:
        _req(out, "out", torch.bfloat16, 2)
        if out.shape[1] != H:
            raise ValueError(f"out must be [R, {H}], got {tuple(out.shape)}")
    _launch(dev, "moe_permute", _ptr(x), _ptr(row_of_slot), T, k, out.shape[0], H, _ptr(out))
    return out


def moe_permute_fp8(x, row_of_slot, *, codes=None, scales=None):
    """e4m3 codes [R, H] and f32 row scales [R] of moe_permute's rows, as
    quantize_rows_fp8 gives them: the operands of gmm_fp8_fwd_q and
    gmm_silu_fp8_q."""
    if codes is None and scales is None:
        r = (_calls or _plain()).permute_fp8(x, row_of_slot)
        if r is not None:
            return r
    dev, T, k, H = _slots(x, "x", row_of_slot, True, codes, scales)
    R = T * k if codes is None else codes.shape[0]
    codes = _out(codes, (R, H), torch.uint8, dev, "codes")
    scales = _out(scales, (R,), torch.float32, dev, "scales")
    _launch(dev, "moe_permute_fp8", _ptr(x), _ptr(row_of_slot), T, k, R, H, _ptr(codes), _ptr(scales))
    return codes, scales


def moe_combine(y, row_of_slot, weights=None, *, out=None):
    """bf16 [T, H]: the sum of each token's rows of y [R, H] with its weights
    [T, k]; without weights the plain sum, moe_permute's gradient."""
    if out is None:
        out = (_calls or _plain()).combine(y, row_of_slot, weights)
        if out is not None:
            return out
    dev, T, k, H = _slots(y, "y", row_of_slot, False, weights, out)
    if weights is not None:
        _req_slots(weights, "weights", torch.float32, T, k)
    out = _out(out, (T, H), torch.bfloat16, dev, "out")
    _launch(dev, "moe_combine", _ptr(y), _ptr(row_of_slot), _ptr(weights), T, k, y.shape[0], H, _ptr(out))
    return out


def moe_combine_bwd(dout, y, row_of_slot, weights, *, dy=None, dweights=None):
    """moe_combine's gradients from dout [T, H]: (dy bf16 [R, H], dweights f32
    [T, k]).  Rows of dy that no slot names are left as they are."""
    if dy is None and dweights is None:
        r = (_calls or _plain()).combine_bwd(dout, y, row_of_slot, weights)
        if r is not None:
            return r
    dev, T, k, H = _slots(dout, "dout", row_of_slot, True, y, weights, dy, dweights)
    _req(y, "y", torch.bfloat16, 2)
    if y.shape[1] != H:
        raise ValueError(f"y must be [R, {H}], got {tuple(y.shape)}")
    _req_slots(weights, "weights", torch.float32, T, k)
    dy = _out(dy, tuple(y.shape), torch.bfloat16, dev, "dy")
    dweights = _out(dweights, (T, k), torch.float32, dev, "dweights")
    _launch(dev, "moe_combine_bwd", _ptr(dout), _ptr(y), _ptr(row_of_slot), _ptr(weights), T, k, y.shape[0], H, _ptr(dy),
            _ptr(dweights))
    return dy, dweights


# --------------------------------------------------------------------------- balance losses

class MoeBalance(NamedTuple):
    """What moe_balance_loss returns."""
    losses: torch.Tensor       # float32 [2]: balance (1 for an even load), mean square of the logits' log-sum-exp
    counts: torch.Tensor       # int32 [E]
    probs: torch.Tensor        # float32 [E], mean over the tokens that count
    tokens: torch.Tensor       # int32 [1], how many count


def _req_vector(t, name, dtype, n):
    _req(t, name, dtype, 1)
    if t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}], got {tuple(t.shape)}")


def moe_balance_loss(logits, ids=None, *, counts=None, workspace=None):
    """The balance losses of router logits [T, E] (float32 or bfloat16; a token
    whose logits are all -inf does not count): a MoeBalance.  The experts' loads
    are counted from ``ids`` [T, k] (moe_route's), or given as ``counts`` int32
    [E], for example moe_route's group_sizes summed over several ranks."""
    if workspace is None:
        r = (_calls or _plain()).balance(logits, ids, counts)
        if r is not None:
            return MoeBalance._make(r)
    _req_logits(logits)
    T, E = logits.shape
    _req_i32(E, "the number of experts")
    if (ids is None) == (counts is None):
        raise ValueError("either ids or counts must be given")
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, 1)
    dev = _same_device(logits, ids, counts, workspace)
    k = 1
    if ids is None:
        _req_vector(counts, "counts", torch.int32, E)
    else:
        _req(ids, "ids", torch.int32, 2)
        k = ids.shape[1]
        _req_i32(k, "k")
        if ids.shape[0] != T:
            raise ValueError(f"ids must be [{T}, k], got {tuple(ids.shape)}")
        counts = torch.empty((E,), dtype=torch.int32, device=dev)
    losses, probs = torch.empty((2,), device=dev), torch.empty((E,), device=dev)
    tokens = torch.empty((1,), dtype=torch.int32, device=dev)
    ws, need = _workspace(OP_BALANCE, T, E, k, 1, dev, tile_m=0, workspace=workspace)
    # an empty tensor's pointer is NULL, which would make counts an input: any other stands for no ids
    ids_ptr = None if ids is None else _ptr(ids) or _ptr(tokens)
    _launch(dev, "moe_balance_loss", _ptr(logits), LOGIT_DTYPES[logits.dtype], ids_ptr, T, E, k, _ptr(losses),
            _ptr(counts), _ptr(probs), _ptr(tokens), _ptr(ws), need)
    return MoeBalance(losses, counts, probs, tokens)


def moe_balance_loss_bwd(dlosses, logits, counts, tokens, *, add=None, out=None):
    """The logits' gradient, in their type [T, E], of moe_balance_loss's losses
    weighted by dlosses float32 [2], from the forward's counts and tokens.
    ``add`` (for example moe_route_bwd's result) is added before the rounding;
    ``out`` may be ``add`` itself."""
    if out is None:
        r = (_calls or _plain()).balance_bwd(dlosses, logits, counts, tokens, add)
        if r is not None:
            return r
    _req_logits(logits)
    T, E = logits.shape
    _req_i32(E, "the number of experts")
    _req_vector(dlosses, "dlosses", torch.float32, 2)
    _req_vector(counts, "counts", torch.int32, E)
    _req_vector(tokens, "tokens", torch.int32, 1)
    dev = _same_device(dlosses, logits, counts, tokens, add, out)
    if add is not None:
        add = _out(add, (T, E), logits.dtype, dev, "add")
    out = _out(out, (T, E), logits.dtype, dev, "out")
    _launch(dev, "moe_balance_loss_bwd", _ptr(dlosses), _ptr(logits), LOGIT_DTYPES[logits.dtype], _ptr(counts),
            _ptr(tokens), T, E, _ptr(add), _ptr(out))
    return out


# --------------------------------------------------------------------------- AdamW, weight codes

class _AdamW(ctypes.Structure):
    """fp8gmm_adamw of the header."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
        [("step", _I64), ("lr_dev", _P), ("step_dev", _P), ("grad_scale", _P)]


STATE_BLOCK = 256      # consecutive elements that share one scale of an 8-bit state


def adamw_8bit_states(params):
    """Zero states of adamw_step_8bit for a list of parameters: two lists of
    (codes uint8 of the parameter's shape, scales float32 [ceil(size / 256)])."""
    def zeros(p):
        return (torch.zeros(p.shape, dtype=torch.uint8, device=p.device),
                torch.zeros(-(-p.numel() // STATE_BLOCK), device=p.device))
    return [zeros(p) for p in params], [zeros(p) for p in params]


def _number_or_device(v, name, dtype, dev):
    """(host number, device pointer) of a number or a tensor of one."""
    if not isinstance(v, torch.Tensor):
        return v, None
    if v.dtype != dtype:
        raise TypeError(f"{name} must be a number or a {dtype} tensor, got {v.dtype}")
    if v.numel() != 1:
        raise ValueError(f"{name} must hold one number, got shape {tuple(v.shape)}")
    if v.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {v.device}")
    return 0, v.data_ptr()


def _adamw(name, params, grads, states, held, lr, step, betas, eps, weight_decay, grad_scale, seed):
    lists = [list(params), list(grads)] + [list(s) for s in states]
    n = len(lists[0])
    if any(len(l) != n for l in lists):
        raise ValueError(f"the lists must have one length, got {[len(l) for l in lists]}")
    if n == 0:
        return
    columns, named = lists[:2], ["params", "grads"]
    if held:
        for l, what in zip(lists[2:], ("exp_avgs", "exp_avg_roots")):
            if any(not isinstance(s, (tuple, list)) or len(s) != 2 for s in l):
                raise TypeError(f"{what} must hold pairs (codes, scales)")
            columns, named = columns + [[s[0] for s in l], [s[1] for s in l]], named + [what + " codes", what + " scales"]
    else:
        columns, named = lists, named + ["exp_avgs", "exp_avg_sqs"]
    for l, what in zip(columns, named):
        for t in l:
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{what} must hold torch.Tensors")
            if what in ("params", "grads"):
                if t.dtype not in LOGIT_DTYPES or t.dtype != l[0].dtype:
                    raise TypeError(f"{what} must all be float32 or all bfloat16, got {t.dtype}")
                dtype = t.dtype
            else:
                dtype = torch.uint8 if what.endswith("codes") else torch.float32
            _req(t, what, dtype, t.dim())
    for i, p in enumerate(columns[0]):
        for l, what in zip(columns[1:], named[1:]):
            want = (-(-p.numel() // STATE_BLOCK),) if what.endswith("scales") else tuple(p.shape)
            if tuple(l[i].shape) != want:
                raise ValueError(f"{what}[{i}] must be {want}, got {tuple(l[i].shape)}")
    dev = _same_device(*(t for l in columns for t in l))
    how = _AdamW(beta1=float(betas[0]), beta2=float(betas[1]), eps=float(eps), weight_decay=float(weight_decay))
    lr, how.lr_dev = _number_or_device(lr, "lr", torch.float32, dev)
    step, how.step_dev = _number_or_device(step, "step", torch.int64, dev)
    if grad_scale is not None:
        if not isinstance(grad_scale, torch.Tensor):
            raise TypeError("grad_scale must be a torch.Tensor")
        _, how.grad_scale = _number_or_device(grad_scale, "grad_scale", torch.float32, dev)
    how.lr, step = float(lr), int(step)
    if how.step_dev is None and not 1 <= step < 1 << 63:
        raise ValueError(f"step must be at least 1, got {step}")
    how.step = step
    rates = [how.lr, how.eps, how.weight_decay]
    if not all(0 <= v < float("inf") for v in rates) or not all(0 <= b < 1 for b in (how.beta1, how.beta2)):
        raise ValueError(f"lr, eps and weight_decay must be finite and not negative, betas in [0, 1): got {rates}, {betas}")
    if how.eps != 0 and not 2.0 ** -126 <= how.eps <= 2.0 ** 126:
        raise ValueError(f"eps must be 0 or from 2^-126 to 2^126, got {eps}")
    if max(how.lr * how.weight_decay, how.lr / (1 - how.beta1)) > torch.finfo(torch.float32).max:
        raise ValueError(f"lr * weight_decay and lr / (1 - beta1) must be float32 numbers, got lr {how.lr}")
    if held and not 0 <= seed < 1 << 64:
        raise ValueError(f"seed must fit 64 bits without a sign, got {seed}")
    pointers = [(_P * n)(*(t.data_ptr() for t in l)) for l in columns]
    sizes = (_I64 * n)(*(p.numel() for p in columns[0]))
    p, g = LOGIT_DTYPES[columns[0][0].dtype], LOGIT_DTYPES[columns[1][0].dtype]
    _launch(dev, name, n, sizes, pointers[0], p, pointers[1], g, *pointers[2:], *((seed,) if held else ()),
            ctypes.byref(how))
    # a graph that has saved a parameter notices that it changed
    torch.autograd.graph.increment_version([t for t in columns[0] if not t.is_inference()])


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
               grad_scale=None):
    """One AdamW step over lists of tensors, in place: parameters and gradients
    float32 or bfloat16, states float32.  ``step`` counts from 1.  ``lr`` and
    ``step`` may be tensors of one number on the device (float32, int64), read
    when the kernels run, for captured graphs, with coefficients rounded as those
    of the host's numbers; ``grad_scale`` is such a float32 tensor that multiplies
    the gradients.  Tensors may be pieces of one buffer, at any element; one may be
    listed once."""
    st = (_calls or _plain()).adamw(params, grads, exp_avgs, exp_avg_sqs, lr, step, *betas, eps, weight_decay,
                                    grad_scale)
    if st is None:
        _adamw("adamw_step", params, grads, (exp_avgs, exp_avg_sqs), False, lr, step, betas, eps, weight_decay,
               grad_scale, 0)
    elif st != OK:
        raise Fp8GmmError("adamw_step", st)


def adamw_step_8bit(params, grads, exp_avgs, exp_avg_roots, *, lr, step, betas=(0.9, 0.999), eps=1e-8,
                    weight_decay=0.01, grad_scale=None, seed=0):
    """adamw_step with states in 8 bits: lists of (codes, scales) as
    adamw_8bit_states makes them, of the first moment and of the second one's
    square root.  Codes are rounded up or down by chance, as ``seed`` and
    ``step`` decide: the same call on the same tensors gives the same bits.  The
    mean of the root is kept; the second moment is held some 5 % too high."""
    seed = int(seed)
    st = (_calls or _plain()).adamw8(params, grads, exp_avgs, exp_avg_roots, lr, step, *betas, eps, weight_decay,
                                     grad_scale, seed)
    if st is None:
        _adamw("adamw_step_8bit", params, grads, (exp_avgs, exp_avg_roots), True, lr, step, betas, eps, weight_decay,
               grad_scale, seed)
    elif st != OK:
        raise Fp8GmmError("adamw_step_8bit", st)


def quantize_fp8_weights(w, *, codes=None, scales=None, workspace=None):
    """e4m3 codes u8 [G, K, N] and f32 scales [G, N], one per output channel over
    all K, of master weights w [G, K, N] (float32 or bfloat16): what the FP8
    calls read."""
    if codes is None and scales is None and workspace is None:
        r = (_calls or _plain()).quantize_fp8(w)
        if r is not None:
            return r
    if isinstance(w, torch.Tensor) and w.dtype not in LOGIT_DTYPES:
        raise TypeError(f"w must be float32 or bfloat16, got {w.dtype}")
    _req(w, "w", getattr(w, "dtype", None), 3)
    G, K, N = w.shape
    _req_i32(G, "the number of experts")
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, 1)
    dev = _same_device(w, codes, scales, workspace)
    codes = _out(codes, (G, K, N), torch.uint8, dev, "codes")
    scales = _out(scales, (G, N), torch.float32, dev, "scales")
    ws, need = _workspace(OP_QUANT_WEIGHTS, 0, K, N, G, dev, tile_m=LOGIT_DTYPES[w.dtype], workspace=workspace)
    _launch(dev, "quantize_fp8_weights", _ptr(w), LOGIT_DTYPES[w.dtype], K, N, G, _ptr(codes), _ptr(scales), _ptr(ws),
            need)
    return codes, scales


# --------------------------------------------------------------------------- MXFP4

def quantize_mxfp4_weights(w, *, codes=None, scales=None):
    """MXFP4 codes u8 [G, N, K/2] and scales u8 [G, K/128, N, 4] of weights
    w bf16 [G, K, N], in blocks of 32 along K."""
    if codes is None and scales is None:
        r = (_calls or _plain()).quantize_weights(w)
        if r is not None:
            return r
    _req(w, "w", torch.bfloat16, 3)
    G, K, N = w.shape
    _req_i32(G, "the number of experts")
    dev = w.device
    codes = _out(codes, (G, N, K // 2), torch.uint8, dev, "codes")
    scales = _out(scales, (G, K // 128, N, 4), torch.uint8, dev, "scales")
    _same_device(w, codes, scales)
    _launch(dev, "quantize_mxfp4_weights", _ptr(w), K, N, G, _ptr(codes), _ptr(scales))
    return codes, scales


def _mxfp4_shapes(codes, scales):
    _req(codes, "codes", torch.uint8, 3)
    _req(scales, "scales", torch.uint8, 4)
    G, N, half = codes.shape
    K = 2 * half
    _req_i32(G, "the number of experts")
    if tuple(scales.shape) != (G, K // 128, N, 4):
        raise ValueError(f"scales must be [{G}, {K // 128}, {N}, 4] for codes {tuple(codes.shape)}, "
                         f"got {tuple(scales.shape)}")
    return G, K, N


def dequantize_mxfp4(codes, scales, *, out=None):
    """The values bf16 [G, N, K] of MXFP4 codes [G, N, K/2] and scales
    [G, K/128, N, 4]."""
    if out is None:
        out = (_calls or _plain()).values(codes, scales)
        if out is not None:
            return out
    G, K, N = _mxfp4_shapes(codes, scales)
    dev = _same_device(codes, scales)
    out = _out(out, (G, N, K), torch.bfloat16, dev, "out")
    _same_device(codes, out)
    _launch(dev, "dequantize_mxfp4", _ptr(codes), _ptr(scales), K, N, G, _ptr(out))
    return out


def _mxfp4_product(name, x, codes, scales, group_sizes, slot_of_row, topk, out, dev_status, workspace, swiglu):
    topk = int(topk)
    _req_i32(topk, "topk")
    if out is None and workspace is None and dev_status is None:
        out = (_calls or _plain()).product(x, codes, scales, group_sizes, slot_of_row, topk, swiglu)
        if out is not None:
            return out
    _req(x, "x", torch.bfloat16, 2)
    G, K, N = _mxfp4_shapes(codes, scales)
    _req(group_sizes, "group_sizes", torch.int32, 1)
    T = x.shape[0]
    M = T
    if slot_of_row is not None:
        _req(slot_of_row, "slot_of_row", torch.int32, 1)
        M = slot_of_row.shape[0]
    if x.shape[1] != K or group_sizes.shape[0] != G:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)} codes {tuple(codes.shape)} "
                         f"group_sizes {tuple(group_sizes.shape)}")
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, getattr(dev_status, "ndim", 1))
        if dev_status.numel() == 0:
            raise ValueError("dev_status must hold a word")
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, 1)
    dev = _same_device(x, codes, scales, group_sizes, slot_of_row, dev_status, workspace)
    out = _out(out, (M, N // 2 if swiglu else N), torch.bfloat16, dev, "out")
    _same_device(x, out)
    ws, need = _workspace(OP_MXFP4, T, K, N, G, dev, tile_m=0, workspace=workspace)
    _launch(dev, name, _ptr(x), _ptr(codes), _ptr(scales), _ptr(group_sizes), _ptr(slot_of_row), topk, T, M, K, N, G,
            _ptr(out), _ptr(ws), need, _ptr(dev_status))
    return out


def gmm_mxfp4_fwd(x, codes, scales, group_sizes, *, slot_of_row=None, topk=1, out=None, dev_status=None,
                  workspace=None):
    """Grouped product on 4-bit operands: x bf16 [T, K] is quantized to MXFP4 a
    token, row r reads token slot_of_row[r] // topk (row r without slot_of_row);
    bf16 [M, N]."""
    return _mxfp4_product("gmm_mxfp4_fwd", x, codes, scales, group_sizes, slot_of_row, topk, out, dev_status,
                          workspace, False)


def gmm_silu_mxfp4(x, codes, scales, group_sizes, *, slot_of_row=None, topk=1, out=None, dev_status=None,
                   workspace=None):
    """gmm_mxfp4_fwd with SwiGLU over the columns [gate | up]; bf16 [M, N/2]."""
    return _mxfp4_product("gmm_silu_mxfp4", x, codes, scales, group_sizes, slot_of_row, topk, out, dev_status,
                          workspace, True)
