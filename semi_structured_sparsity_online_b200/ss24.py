"""ctypes binding of ``libss24.so`` (declared in ``include/ss24.h``).

Argument marshalling only: every step of the pass runs in the library's CUDA
kernels. PyTorch supplies device memory (outputs are allocated as torch
tensors) and the current CUDA stream. The raw C functions are available as
``lib().ss24_*``; the helpers below wrap them for torch tensors.

The library must have been built (``semi_structured_sparsity_online_b200.build``
or ``__graft_entry__.build()``); loading fails loudly otherwise. There is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libss24.so")

# enums (include/ss24.h)
OK = 0
STATUS_NAMES = {0: "SS24_OK", 1: "SS24_ERR_NULL", 2: "SS24_ERR_SHAPE", 3: "SS24_ERR_ALIGN",
                4: "SS24_ERR_DTYPE", 5: "SS24_ERR_FORMAT", 6: "SS24_ERR_WORKSPACE", 7: "SS24_ERR_CUDA",
                8: "SS24_ERR_ARG"}
STATUS_NAMES_INV = {v: k for k, v in STATUS_NAMES.items()}
BF16, F32 = 0, 1
MAG, WANDA = 0, 1
DENSE, SPARSE_24, SPARSE_48 = 0, 24, 48
FMT_NONE, FMT_FP8, FMT_INT, FMT_NVFP4, FMT_MXFP4 = 0, 1, 2, 3, 4
_FMT = {"none": FMT_NONE, "fp8": FMT_FP8, "int": FMT_INT, "nvfp4": FMT_NVFP4, "mxfp4": FMT_MXFP4}
_SCORE = {"mag": MAG, "wanda": WANDA}


class Format(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("pack4", ctypes.c_int32)]


class Operand(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("axis", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("batch", ctypes.c_int64), ("batch_stride", ctypes.c_int64),
                ("hadamard", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Outputs(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("meta", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("kind", ctypes.c_int32), ("page", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KvBatch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("table_ld", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("max_new", ctypes.c_int64), ("max_len", ctypes.c_int64)]


class HeadRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class SS24Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lib = None
_P = ctypes.c_void_p
_S = ctypes.c_size_t
_OP = ctypes.POINTER(Operand)
_OUT = ctypes.POINTER(Outputs)
_KVC = ctypes.POINTER(KvCache)
_KVB = ctypes.POINTER(KvBatch)
_HR = ctypes.POINTER(HeadRows)

_SIGNATURES = {
    "ss24_workspace_bytes": (ctypes.c_size_t, []),
    "ss24_workspace_init": (ctypes.c_int, [_P, _S, _P]),
    "ss24_workspace_error": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
    "ss24_prune24_compress": (ctypes.c_int, [_OP, ctypes.c_int, _P, _P, _P, _P, _P, _S, _P]),
    "ss24_quantize_fp8": (ctypes.c_int, [_OP, _P, _OUT, _P, _P, _S, _P]),
    "ss24_quantize_int": (ctypes.c_int, [_OP, Format, _OUT, _P, _P, _S, _P]),
    "ss24_quantize_nvfp4": (ctypes.c_int, [_OP, _P, _OUT, _P, _P, _S, _P]),
    "ss24_quantize_mxfp4": (ctypes.c_int, [_OP, _OUT, _P, _P, _S, _P]),
    "ss24_prune24_quant_fused": (ctypes.c_int, [_OP, ctypes.c_int, _P, Format, _P, _OUT, _P, _P, _S, _P]),
    "ss24_prune24_quant_fused_noalloc": (ctypes.c_int, [_OP, ctypes.c_int, _P, Format, _P, _OUT, _P, _P]),
    "ss24_prune48_pairwise_quant_fused": (ctypes.c_int,
                                          [_OP, ctypes.c_int, _P, Format, _P, _OUT, _P, _P, _S, _P]),
    "ss24_error_energy": (ctypes.c_int, [_OP, ctypes.c_int, ctypes.c_int, _P, Format, Format, _P, _P, _P, _P,
                                         _S, _P]),
    "ss24_amax": (ctypes.c_int, [_OP, ctypes.c_int, ctypes.c_int, _P, _P, _P, _S, _P]),
    "ss24_tensor_scale": (ctypes.c_int, [_OP, ctypes.c_int, ctypes.c_int, _P, ctypes.c_int32, _P, _P, _S, _P]),
    "ss24_predicted_ratio": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, _P]),
    "ss24_bits_per_element": (ctypes.c_double, [Format, ctypes.c_int, ctypes.c_int64, ctypes.c_int32]),
    "ss24_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ss24_selfcheck_division": (ctypes.c_int, [ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint32, _P, _P]),
    "ss24_amax_rows": (ctypes.c_int, [_OP, ctypes.c_int, ctypes.c_int, _P, _P, ctypes.c_int32, _P, _P, _S, _P]),
    "ss24_quantize_int_rows": (ctypes.c_int, [_OP, ctypes.c_int, ctypes.c_int, _P, Format, _P, _OUT, _P, _P, _S,
                                              _P]),
    "ss24_dequantize": (ctypes.c_int, [_OP, ctypes.c_int, Format, _OUT, _P, _P]),
    "ss24_hadamard": (ctypes.c_int, [_OP, ctypes.c_int32, _P, _P]),
    "ss24_softmax_prune": (ctypes.c_int, [_OP, ctypes.c_float, ctypes.c_int, Format, _P, _OUT, _P, _P,
                                          ctypes.c_size_t, _P]),
    "ss24_scale_tiles_bytes": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64]),
    "ss24_scale_tiles": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P]),
    "ss24_selfcheck_encoder": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint32,
                                              _P, _P]),
    "ss24_sparse_gemm_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                            _P, _P, _S, _P]),
    "ss24_gemm_int8": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P,
                                      ctypes.c_int32, ctypes.c_int64, _P, _S, _P]),
    "ss24_kv_append": (ctypes.c_int, [_KVC, _KVB, _HR, _HR, _P, _S, _P]),
    "ss24_kv_attention_scratch_bytes": (ctypes.c_int64, [_KVC, _KVB, ctypes.c_int32]),
    "ss24_kv_attention": (ctypes.c_int, [_HR, _KVC, _KVB, ctypes.c_float, ctypes.c_int32, _HR, _P, _P,
                                         ctypes.c_int64, _P, _S, _P]),
    "ss24_encode_e4m3": (ctypes.c_int, [_P, _P, ctypes.c_int64, _P]),
    "ss24_decode_e4m3": (ctypes.c_int, [_P, _P, ctypes.c_int64, _P]),
    "ss24_encode_e2m1": (ctypes.c_int, [_P, _P, ctypes.c_int64, _P]),
    "ss24_decode_e2m1": (ctypes.c_int, [_P, _P, ctypes.c_int64, _P]),
}


def lib():
    """Load libss24.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first "
                               "(python -m semi_structured_sparsity_online_b200.build)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def _check(status: int, where: str):
    if status != OK:
        raise SS24Error(status, where)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_format(fmt="none", bits=8, group=0, pack4=False) -> Format:
    kind = _FMT[fmt] if isinstance(fmt, str) else int(fmt)
    return Format(kind, int(bits), int(group), int(bool(pack4)))


def make_operand(x: torch.Tensor, axis: int = 1, rows=None, k=None, hadamard: int = 0) -> Operand:
    """Operand descriptor of a CUDA tensor. 2-D: one operand; axis 1: x is
    [rows, ld] with k contiguous; axis 0: x is [k, ld] holding A[r][c] at
    x[c][r]. 3-D [B, ., .]: a batch of B such operands (x.stride(0) apart).
    hadamard: 0, or the block of the rotation the pass applies along k first."""
    if x.dtype == torch.bfloat16:
        dt = BF16
    elif x.dtype == torch.float32:
        dt = F32
    else:
        raise TypeError("operand must be bfloat16 or float32")
    if x.dim() not in (2, 3) or x.stride(-1) != 1:
        raise ValueError("operand must be 2-D or 3-D with a contiguous last dimension")
    batch, bstride = (x.shape[0], x.stride(0)) if x.dim() == 3 else (1, 0)
    m = x[0] if x.dim() == 3 else x
    if axis == 1:
        r = m.shape[0] if rows is None else rows
        kk = m.shape[1] if k is None else k
    else:
        kk = m.shape[0] if k is None else k
        r = m.shape[1] if rows is None else rows
    return Operand(x.data_ptr(), dt, axis, r, kk, m.stride(0), batch, bstride, int(hadamard), 0)


class Workspace:
    """Device workspace for the library's calls (allocated by torch, cleared once)."""

    def __init__(self, device=None, stream=None):
        n = lib().ss24_workspace_bytes()
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buf.data_ptr()) % 256
        self.tensor = self.buf[off:off + n]
        self.nbytes = n
        _check(lib().ss24_workspace_init(self.ptr, n, _stream(stream)), "ss24_workspace_init")

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    def error(self, stream=None) -> int:
        code = ctypes.c_int32(0)
        _check(lib().ss24_workspace_error(self.ptr, ctypes.byref(code), _stream(stream)), "ss24_workspace_error")
        return code.value


_default_ws = {}
_graph_ws = []


def default_workspace(device=None) -> Workspace:
    """The device's workspace for calls that name none, made by the first of them. Make it before a capture: a call
    captured without one gets a workspace of its own, part of the graph, whose error word every replay clears."""
    dev = torch.device(device or "cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    ws = _default_ws.get(dev)
    if ws is None:
        ws = Workspace(dev)
        if torch.cuda.is_current_stream_capturing():
            _graph_ws.append(ws)  # the graph's calls use it, on whichever stream, as long as the graph lives
            return ws
        # calls on other streams find it cleared
        torch.cuda.current_stream().synchronize()
        _default_ws[dev] = ws
    return ws


def _alloc_outputs(x_rows, k, pattern, fmt: Format, in_dtype, device, batch=None):
    """Output tensors of a pass; with `batch` every output gets a leading
    [batch] dimension (the per-operand outputs packed one after the other)."""
    sparse = pattern != DENSE
    n = k // 2 if sparse else k
    lead = () if batch is None else (batch,)
    out = {}

    def empty(shape, dtype):
        return torch.empty(lead + shape, dtype=dtype, device=device)

    if fmt.kind == FMT_NONE:
        out["values"] = empty((x_rows, n), in_dtype)
    elif fmt.kind == FMT_FP8:
        out["values"] = empty((x_rows, n), torch.uint8)
    elif fmt.kind == FMT_INT:
        if fmt.pack4:
            out["values"] = empty((x_rows, n // 2), torch.uint8)
        else:
            out["values"] = empty((x_rows, n), torch.int16 if fmt.bits > 8 else torch.int8)
        g = fmt.group or n
        out["scales"] = empty((x_rows, n // g), torch.float32)
    elif fmt.kind in (FMT_NVFP4, FMT_MXFP4):
        out["values"] = empty((x_rows, n // 2), torch.uint8)
        blk = 16 if fmt.kind == FMT_NVFP4 else 32
        out["scales"] = empty((x_rows, n // blk), torch.uint8)
    if fmt.kind in (FMT_FP8, FMT_NVFP4):
        out["tensor_scale"] = empty((1,), torch.float32) if batch is None else torch.empty(
            (batch,), dtype=torch.float32, device=device)
    if sparse:
        out["meta"] = empty((x_rows, k // (16 if pattern == SPARSE_48 else 8)), torch.uint8)
    return out


def _lead(op):
    return None if op.batch <= 1 and op.batch_stride == 0 else op.batch


def _energy(op, device):
    b = _lead(op)
    return torch.zeros((4,) if b is None else (b, 4), dtype=torch.float64, device=device)


def run(x: torch.Tensor, pattern=SPARSE_24, fmt="none", bits=8, group=0, pack4=False, score="mag",
        col_norms=None, tensor_scale=None, energy=True, axis=1, ws=None, stream=None, out=None, hadamard=0):
    """One pass through the matching C entry point. Returns a dict of output
    tensors (``values``, ``scales``, ``tensor_scale``, ``meta``) and ``energy``
    (float64[4] on the device: e_total, e_prune, e_quant, e_quant_dense). A
    3-D x is a batch: every output and the energies get a leading [B].
    hadamard=b rotates x along k in the pass first (block Hadamard of b, the
    result rounded to bf16; bf16 input, magnitude score), and so do the amax
    passes behind a derived tensor scale."""
    f = make_format(fmt, bits, group, pack4)
    op = make_operand(x, axis, hadamard=hadamard)
    sc = _SCORE[score] if isinstance(score, str) else int(score)
    if out is None:
        out = _alloc_outputs(op.rows, op.k, pattern, f, x.dtype, x.device, _lead(op))
    e = _energy(op, x.device) if energy is True else energy
    if e is not None and e is not False:
        out["energy"] = e
    else:
        e = None
    ws = ws or default_workspace(x.device)
    o = Outputs(*(_ptr(out.get(key)) for key in ("values", "scales", "tensor_scale", "meta")))
    s = _stream(stream)
    L = lib()
    if pattern == DENSE:
        if f.kind == FMT_FP8:
            st = L.ss24_quantize_fp8(ctypes.byref(op), _ptr(tensor_scale), ctypes.byref(o), _ptr(e), ws.ptr,
                                     ws.nbytes, s)
        elif f.kind == FMT_INT:
            st = L.ss24_quantize_int(ctypes.byref(op), f, ctypes.byref(o), _ptr(e), ws.ptr, ws.nbytes, s)
        elif f.kind == FMT_NVFP4:
            st = L.ss24_quantize_nvfp4(ctypes.byref(op), _ptr(tensor_scale), ctypes.byref(o), _ptr(e), ws.ptr,
                                       ws.nbytes, s)
        elif f.kind == FMT_MXFP4:
            st = L.ss24_quantize_mxfp4(ctypes.byref(op), ctypes.byref(o), _ptr(e), ws.ptr, ws.nbytes, s)
        else:
            raise ValueError("dense pattern needs a quantization format")
        _check(st, "ss24_quantize")
    elif pattern == SPARSE_24 and f.kind == FMT_NONE and tensor_scale is None:
        _check(L.ss24_prune24_compress(ctypes.byref(op), sc, _ptr(col_norms), _ptr(out["values"]),
                                       _ptr(out["meta"]), _ptr(e), ws.ptr, ws.nbytes, s), "ss24_prune24_compress")
    else:
        fn = L.ss24_prune24_quant_fused if pattern == SPARSE_24 else L.ss24_prune48_pairwise_quant_fused
        _check(fn(ctypes.byref(op), sc, _ptr(col_norms), f, _ptr(tensor_scale), ctypes.byref(o), _ptr(e),
                  ws.ptr, ws.nbytes, s), "ss24_prune_quant_fused")
    return out


def error_energy(x, pattern=SPARSE_24, sparse_fmt=("none",), dense_fmt=("int", 8, 0), score="mag",
                 col_norms=None, sparse_scale=None, dense_scale=None, axis=1, ws=None, stream=None, energy=None,
                 hadamard=0):
    """Read-only energy pass; returns float64[4] (or [B, 4]) on the device."""
    sf = make_format(*sparse_fmt) if isinstance(sparse_fmt, tuple) else sparse_fmt
    df = make_format(*dense_fmt) if isinstance(dense_fmt, tuple) else dense_fmt
    op = make_operand(x, axis, hadamard=hadamard)
    e = energy if energy is not None else _energy(op, x.device)
    ws = ws or default_workspace(x.device)
    _check(lib().ss24_error_energy(ctypes.byref(op), pattern, _SCORE[score] if isinstance(score, str) else score,
                                   _ptr(col_norms), sf, df, _ptr(sparse_scale), _ptr(dense_scale), _ptr(e), ws.ptr,
                                   ws.nbytes, _stream(stream)), "ss24_error_energy")
    return e


def amax(x, pattern=SPARSE_24, score="mag", col_norms=None, axis=1, ws=None, stream=None, hadamard=0):
    op = make_operand(x, axis, hadamard=hadamard)
    out = torch.empty(max(op.batch, 1), dtype=torch.float32, device=x.device)
    ws = ws or default_workspace(x.device)
    _check(lib().ss24_amax(ctypes.byref(op), pattern, _SCORE[score] if isinstance(score, str) else score,
                           _ptr(col_norms), _ptr(out), ws.ptr, ws.nbytes, _stream(stream)), "ss24_amax")
    return out


def tensor_scale(x, fmt="fp8", pattern=SPARSE_24, score="mag", col_norms=None, axis=1, ws=None, stream=None,
                 out=None, hadamard=0):
    """The per-tensor scale (FP8: amax / 448, NVFP4: amax / 2688) as a device
    float32[1] (float32[B] for a batch)."""
    op = make_operand(x, axis, hadamard=hadamard)
    out = out if out is not None else torch.empty(max(op.batch, 1), dtype=torch.float32, device=x.device)
    ws = ws or default_workspace(x.device)
    _check(lib().ss24_tensor_scale(ctypes.byref(op), pattern, _SCORE[score] if isinstance(score, str) else score,
                                   _ptr(col_norms), _FMT[fmt] if isinstance(fmt, str) else fmt, _ptr(out), ws.ptr,
                                   ws.nbytes, _stream(stream)), "ss24_tensor_scale")
    return out


def amax_rows(x, pattern=DENSE, score="mag", col_norms=None, scale_fmt=None, ws=None, stream=None, out=None,
              scale_out=None, hadamard=0):
    """Per-row amax of the values a pass with this pattern / score quantizes,
    float32 [rows] (or [B, rows]) on the device, and, with scale_fmt ("fp8" or
    "nvfp4"), the per-tensor scale from the same read: returns (rows, scale)."""
    op = make_operand(x, 1, hadamard=hadamard)
    lead = _lead(op)
    shape = (op.rows,) if lead is None else (lead, op.rows)
    out = out if out is not None else torch.empty(shape, dtype=torch.float32, device=x.device)
    if scale_fmt is not None and scale_out is None:
        scale_out = torch.empty(max(op.batch, 1), dtype=torch.float32, device=x.device)
    kind = 0 if scale_fmt is None else (_FMT[scale_fmt] if isinstance(scale_fmt, str) else int(scale_fmt))
    ws = ws or default_workspace(x.device)
    _check(lib().ss24_amax_rows(ctypes.byref(op), pattern, _SCORE[score] if isinstance(score, str) else score,
                                _ptr(col_norms), _ptr(out), kind, _ptr(scale_out), ws.ptr, ws.nbytes,
                                _stream(stream)), "ss24_amax_rows")
    return out, scale_out


def run_int_rows(x, row_amax, pattern=DENSE, bits=8, pack4=False, score="mag", col_norms=None, energy=True,
                 ws=None, stream=None, out=None, hadamard=0):
    """INT-b with one scale per row from a given per-row amax (ss24_quantize_int_rows);
    returns the same dict as run()."""
    f = make_format("int", bits, 0, pack4)
    op = make_operand(x, 1, hadamard=hadamard)
    if out is None:
        out = _alloc_outputs(op.rows, op.k, pattern, f, x.dtype, x.device, _lead(op))
    e = _energy(op, x.device) if energy is True else energy
    if e is not None and e is not False:
        out["energy"] = e
    else:
        e = None
    ws = ws or default_workspace(x.device)
    o = Outputs(*(_ptr(out.get(key)) for key in ("values", "scales", "tensor_scale", "meta")))
    _check(lib().ss24_quantize_int_rows(ctypes.byref(op), pattern, _SCORE[score] if isinstance(score, str) else score,
                                        _ptr(col_norms), f, _ptr(row_amax), ctypes.byref(o), _ptr(e), ws.ptr,
                                        ws.nbytes, _stream(stream)), "ss24_quantize_int_rows")
    return out


def dequantize(out, rows, k, pattern=SPARSE_24, fmt="none", bits=8, group=0, pack4=False, dtype=torch.bfloat16,
               batch=None, stream=None, xhat=None):
    """The dense float32 operand [rows, k] (or [B, rows, k]) that the outputs of a
    pass (the dict run() returns) stand for: dequantized values on kept
    positions, zero on dropped ones."""
    f = make_format(fmt, bits, group, pack4)
    dev = out["values"].device
    op = Operand(None, BF16 if dtype == torch.bfloat16 else F32, 1, rows, k, k, batch or 0, 0)
    shape = (rows, k) if batch is None else (batch, rows, k)
    xhat = xhat if xhat is not None else torch.empty(shape, dtype=torch.float32, device=dev)
    o = Outputs(*(_ptr(out.get(key)) for key in ("values", "scales", "tensor_scale", "meta")))
    _check(lib().ss24_dequantize(ctypes.byref(op), pattern, f, ctypes.byref(o), _ptr(xhat), _stream(stream)),
           "ss24_dequantize")
    return xhat


def softmax_prune(s: torch.Tensor, alpha: float, pattern=SPARSE_24, fmt="fp8", bits=8, group=0, pack4=False,
                  tensor_scale=None, energy=True, ws=None, stream=None, out=None):
    """P = softmax(alpha * s) per row, pruned / quantized in the same pass
    (ss24_softmax_prune): the same dict as run() for the bf16 operand P, which
    is never stored. s: logits [rows, keys] or [B, rows, keys], bf16 or fp32."""
    f = make_format(fmt, bits, group, pack4)
    op = make_operand(s, 1)
    if out is None:
        out = _alloc_outputs(op.rows, op.k, pattern, f, torch.bfloat16, s.device, _lead(op))
    e = _energy(op, s.device) if energy is True else energy
    if e is not None and e is not False:
        out["energy"] = e
    else:
        e = None
    ws = ws or default_workspace(s.device)
    o = Outputs(*(_ptr(out.get(key)) for key in ("values", "scales", "tensor_scale", "meta")))
    _check(lib().ss24_softmax_prune(ctypes.byref(op), float(alpha), pattern, f, _ptr(tensor_scale), ctypes.byref(o),
                                    _ptr(e), ws.ptr, ws.nbytes, _stream(stream)),
           "ss24_softmax_prune")
    return out


def hadamard(x: torch.Tensor, block: int, out=None, stream=None):
    """Block Hadamard rotation of x [rows, k] or [B, rows, k] (bf16 or fp32,
    k contiguous) along k (ss24_hadamard): fp32 of the same shape, packed."""
    op = make_operand(x, 1)
    out = out if out is not None else torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _check(lib().ss24_hadamard(ctypes.byref(op), int(block), _ptr(out), _stream(stream)), "ss24_hadamard")
    return out


def scale_tiles(scales, rows, cols, batch=None, out=None, stream=None):
    """NVFP4 / MXFP4 scale bytes (uint8 [rows, cols] or [B, rows, cols] on the
    device, packed) in the block-scaled MMA's 128 x 4 tile layout
    (ss24_scale_tiles): uint8 [B * ss24_scale_tiles_bytes(rows, cols)]."""
    nb = batch or 1
    per = lib().ss24_scale_tiles_bytes(rows, cols)
    if per < 0:
        raise ValueError("negative scale matrix size")
    out = out if out is not None else torch.empty(nb * per, dtype=torch.uint8, device=scales.device)
    _check(lib().ss24_scale_tiles(_ptr(scales), rows, cols, batch or 0, _ptr(out), _stream(stream)),
           "ss24_scale_tiles")
    return out


def predicted_ratio(sparse_energy, dense_energy, out=None, stream=None):
    """float64[..., 4] on the device: loss, rel_err_sparse, rel_err_dense, R_hat,
    for each pair of energy records (float64[..., 4], contiguous)."""
    count = sparse_energy.numel() // 4
    r = out if out is not None else torch.empty_like(sparse_energy)
    _check(lib().ss24_predicted_ratio(_ptr(sparse_energy), _ptr(dense_energy), _ptr(r), count, _stream(stream)),
           "ss24_predicted_ratio")
    return r


def sparse_gemm_fp8(a, b, y=None, ws=None, stream=None):
    """Y = s_a s_b A B^T on the tensor cores' 2:4-sparse FP8 MMA
    (ss24_sparse_gemm_fp8). a: the dict of a 2:4 + FP8 pass over [m, k]
    (``values`` [m, k/2], ``meta`` [m, k/8], ``tensor_scale``); b: the dict of a
    dense FP8 pass over [n, k] (``values`` [n, k], ``tensor_scale``). Returns
    float32 [m, n] on the device."""
    m, n, k = a["values"].shape[0], b["values"].shape[0], b["values"].shape[1]
    y = y if y is not None else torch.empty((m, n), dtype=torch.float32, device=a["values"].device)
    ws = ws or default_workspace(a["values"].device)
    _check(lib().ss24_sparse_gemm_fp8(_ptr(a["values"]), _ptr(a["meta"]), _ptr(a["tensor_scale"]),
                                      _ptr(b["values"]), _ptr(b["tensor_scale"]), m, n, k, _ptr(y), ws.ptr,
                                      ws.nbytes, _stream(stream)), "ss24_sparse_gemm_fp8")
    return y


# ---- serving in 8 bits -------------------------------------------------------

# These wrappers sit on the path of a decode step, where a kernel takes a few
# microseconds: they check with few attribute reads, enter no context that is
# already current and ask for the stream's raw handle only.

# The private forms are faster; a build of torch without CUDA lacks them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _same_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on different devices: {t.device} and index {index}")


def _enqueue(index, stream, name, *args):
    """The C call `name`(*args, stream) with device `index` current, on `stream`
    or that device's current stream."""
    if index < 0:
        raise ValueError(f"{name} needs CUDA tensors")
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if _current_device() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st:
        raise SS24Error(st, name)


def _workspace(ws, t):
    if ws is not None:
        return ws
    ws = _default_ws.get(t.device)
    if ws is None:
        with torch.cuda.device(t.device):
            ws = default_workspace(t.device)
    return ws


def _int8_rows(d, name):
    """Codes and scales of a dense INT8 operand with one scale per row."""
    if d.get("meta") is not None:
        raise ValueError(f"{name} must be dense: it has the metadata of a sparse pass")
    v, s = d["values"], d["scales"]
    if v.dtype != torch.int8 or v.dim() != 2 or not v.is_contiguous():
        raise ValueError(f"{name}['values'] must be contiguous int8 [rows, k]")
    if s.dtype != torch.float32 or s.numel() != v.shape[0] or not s.is_contiguous():
        raise ValueError(f"{name}['scales'] must be contiguous float32, one per row")
    return v, s


def gemm_int8(a, b, dtype=torch.bfloat16, y=None, ws=None, stream=None):
    """Y = diag(s_a) A B^T diag(s_b) on the INT8 tensor cores (ss24_gemm_int8).
    a, b: the dicts of dense INT8 passes with one scale per row over [m, k]
    tokens and [n, k] channels (``values`` int8, ``scales`` float32 [rows, 1]).
    Returns [m, n] in `dtype` (bfloat16 or float32), or fills `y` (its dtype;
    the columns contiguous, any row stride)."""
    if stream is not None and y is None and stream != torch.cuda.current_stream(stream.device):
        with torch.cuda.stream(stream):  # what is allocated here belongs to the stream that uses it
            return gemm_int8(a, b, dtype, None, ws)
    av, sa = _int8_rows(a, "a")
    bv, sb = _int8_rows(b, "b")
    (m, k), (n, kb) = av.shape, bv.shape
    if kb != k:
        raise ValueError("a and b differ in k")
    if y is None:
        if dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise TypeError("y must be bfloat16 or float32")
        y, ld = av.new_empty((m, n), dtype=dtype), n
    else:
        if y.dtype is not torch.bfloat16 and y.dtype is not torch.float32:
            raise TypeError("y must be bfloat16 or float32")
        if tuple(y.shape) != (m, n) or (n > 1 and y.stride(1) != 1) or (m > 1 and y.stride(0) < n):
            raise ValueError("y must be [m, n] with contiguous columns and rows that do not overlap")
        ld = max(y.stride(0), n)
    index = av.get_device()
    _same_device(index, sa, bv, sb, y)
    ws = _workspace(ws, av)
    _enqueue(index, stream, "ss24_gemm_int8", av.data_ptr(), sa.data_ptr(), bv.data_ptr(), sb.data_ptr(), m, n, k,
             y.data_ptr(), F32 if y.dtype is torch.float32 else BF16, ld, ws.tensor.data_ptr(), ws.nbytes)
    return y


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_KV_DTYPE = {"int": (torch.int8, FMT_INT), "fp8": (torch.uint8, FMT_FP8)}


def kv_cache(pages, kv_heads, head_dim, page=64, fmt="int", device=None):
    """An empty 8-bit paged cache (ss24_kv_cache) as a dict: codes ``k``, ``v``
    [pages, kv_heads, page, head_dim] (int8 for "int", uint8 E4M3 for "fp8"),
    ``k_scales``, ``v_scales`` float32 [pages, kv_heads], ``page`` and ``fmt``."""
    if fmt not in _KV_DTYPE:
        raise ValueError("the cache's format is 'int' (8 bits) or 'fp8'")
    dev = torch.device(device or "cuda")
    c = {n: torch.zeros((pages, kv_heads, page, head_dim), dtype=_KV_DTYPE[fmt][0], device=dev) for n in ("k", "v")}
    c.update({n: torch.zeros((pages, kv_heads), dtype=torch.float32, device=dev) for n in ("k_scales", "v_scales")})
    return {**c, "page": page, "fmt": fmt}


def _kv_cache(cache) -> KvCache:
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scales"], cache["v_scales"]
    dt, kind = _KV_DTYPE.get(cache["fmt"], (None, None))
    if dt is None:
        raise ValueError("the cache's format is 'int' (8 bits) or 'fp8'")
    shape, scales = k.shape, ks.shape
    if (k.dtype is not dt or v.dtype is not dt or len(shape) != 4 or v.shape != shape or not k.is_contiguous()
            or not v.is_contiguous()):
        raise ValueError(f"the cache's codes must be contiguous {dt} [pages, kv_heads, page, head_dim]")
    pages, heads, page, d = shape
    if (ks.dtype is not _F32 or vs.dtype is not _F32 or scales != (pages, heads) or vs.shape != scales
            or not ks.is_contiguous() or not vs.is_contiguous()):
        raise ValueError("the cache's scales must be contiguous float32 [pages, kv_heads]")
    if page != cache["page"]:
        raise ValueError("the cache's page is not its codes' third dimension")
    _same_device(k.get_device(), v, ks, vs)
    return KvCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), kind, page, pages, heads, d)


def _kv_batch(cache, tokens, page_table, starts, lengths, max_new, max_len) -> KvBatch:
    if lengths.dtype is not _I32 or lengths.dim() != 1 or not lengths.is_contiguous():
        raise ValueError("lengths must be int32 [seqs]")
    seqs = lengths.numel()
    if starts.dtype is not _I32 or starts.dim() != 1 or starts.numel() != seqs + 1 or not starts.is_contiguous():
        raise ValueError(f"starts must be int32 [{seqs + 1}]")
    if page_table.dtype is not _I32 or page_table.dim() != 2 or page_table.shape[0] != seqs:
        raise ValueError(f"page_table must be int32 [{seqs}, most pages]")
    width = page_table.shape[1]
    ld, col = page_table.stride()
    if seqs <= 1:
        ld = width
    if (width > 1 and col != 1) or ld < width:
        raise ValueError("page_table must have contiguous rows")
    _same_device(cache["k"].get_device(), page_table, starts, lengths)
    room = width * cache["page"]
    max_len = room if max_len is None else int(max_len)
    if max_len > room:
        raise ValueError("max_len does not fit the page table")
    max_new = tokens if max_new is None else min(int(max_new), tokens)
    return KvBatch(page_table.data_ptr(), starts.data_ptr(), lengths.data_ptr(), seqs, ld, tokens, max_new, max_len)


def _head_rows(x, name, head_dim) -> HeadRows:
    dt = x.dtype
    if dt is not _BF16 and dt is not _F32:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if x.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, {head_dim}] with contiguous rows")
    tokens, heads, d = x.shape
    ts, hs, es = x.stride()
    if d != head_dim or es != 1:
        raise ValueError(f"{name} must be [tokens, heads, {head_dim}] with contiguous rows")
    # a stride that only one row would use is free
    return HeadRows(x.data_ptr(), BF16 if dt is _BF16 else F32, heads, ts if tokens > 1 else heads * head_dim,
                    hs if heads > 1 else head_dim)


def kv_append(cache, k, v, page_table, starts, lengths, max_new=None, max_len=None, ws=None, stream=None):
    """New tokens' k, v [tokens, kv_heads, head_dim] (bfloat16 or float32, any
    token and head strides) into the cache (ss24_kv_append), in place; returns
    it. page_table int32 [seqs, most pages], starts int32 [seqs + 1], lengths
    int32 [seqs] (the new tokens included). max_new, max_len: bounds that the
    host knows; by default the loosest ones."""
    c = _kv_cache(cache)
    if k.shape != v.shape:
        raise ValueError("k and v differ in shape")
    kr, vr = _head_rows(k, "k", c.head_dim), _head_rows(v, "v", c.head_dim)
    b = _kv_batch(cache, k.shape[0], page_table, starts, lengths, max_new, max_len)
    index = cache["k"].get_device()
    _same_device(index, k, v)
    ws = _workspace(ws, k)
    _enqueue(index, stream, "ss24_kv_append", c, b, kr, vr, ws.tensor.data_ptr(), ws.nbytes)
    return cache


def kv_attention(q, cache, page_table, starts, lengths, scale=None, causal=True, max_new=None, max_len=None, out=None,
                 lse=False, ws=None, stream=None):
    """Attention of the new tokens' q [tokens, q_heads, head_dim] (bfloat16)
    over the cache (ss24_kv_attention); the sequences as in kv_append. scale:
    1 / sqrt(head_dim) by default. Returns out [tokens, q_heads, head_dim]
    (bfloat16), or (out, lse) with lse=True or an lse tensor (float32 [tokens,
    q_heads]). max_new and max_len choose the kernel and the split of the keys, so
    give them where the host knows them: 64 single tokens over 4000 keys each take
    115 us with max_new=1 and 279 without, a request of 2000 keys in a page table
    for 131072 16 us with max_len=2000 and 35 without."""
    if stream is not None and stream != torch.cuda.current_stream(stream.device):
        # what is allocated here belongs to the stream that uses it
        with torch.cuda.stream(stream):
            return kv_attention(q, cache, page_table, starts, lengths, scale, causal, max_new, max_len, out, lse, ws)
    c = _kv_cache(cache)
    d = c.head_dim
    qr = _head_rows(q, "q", d)
    b = _kv_batch(cache, q.shape[0], page_table, starts, lengths, max_new, max_len)
    heads = qr.heads
    index = cache["k"].get_device()
    _same_device(index, q)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        outr = HeadRows(out.data_ptr(), qr.dtype, heads, heads * d, d)
    else:
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
        outr = _head_rows(out, "out", d)
        _same_device(index, out)
    if lse is True:
        lse = q.new_empty((b.tokens, heads), dtype=_F32)
    elif lse is False or lse is None:
        lse = None
    else:
        if lse.dtype is not _F32 or lse.shape != q.shape[:2] or not lse.is_contiguous():
            raise ValueError("lse must be contiguous float32 [tokens, q_heads]")
        _same_device(index, lse)
    ws = _workspace(ws, q)
    n = (_lib or lib()).ss24_kv_attention_scratch_bytes(c, b, heads)
    scratch = q.new_empty(n, dtype=torch.uint8) if n > 0 else None
    _enqueue(index, None, "ss24_kv_attention", qr, c, b, d ** -0.5 if scale is None else float(scale),
             1 if causal else 0, outr, None if lse is None else lse.data_ptr(),
             None if scratch is None else scratch.data_ptr(), n if n > 0 else 0, ws.tensor.data_ptr(), ws.nbytes)
    return out if lse is None else (out, lse)


def bits_per_element(fmt="none", bits=8, group=0, pattern=SPARSE_24, k=4096, with_scales=False) -> float:
    return lib().ss24_bits_per_element(make_format(fmt, bits, group), pattern, k, int(with_scales))


def status_string(status: int) -> str:
    return lib().ss24_status_string(status).decode()


def selfcheck_division(mode=0, b_first=0, b_count=1 << 23, chunk=1 << 16, stream=None):
    """Mismatches between the kernels' corrected division and IEEE division
    (see ss24_selfcheck_division); returns (count, first mismatch or None)."""
    res = torch.tensor([0, -1], dtype=torch.int64, device="cuda")
    for b0 in range(b_first, b_first + b_count, chunk):
        n = min(chunk, b_first + b_count - b0)
        _check(lib().ss24_selfcheck_division(mode, b0, n, _ptr(res), _stream(stream)), "ss24_selfcheck_division")
    r = res.cpu().numpy().view("uint64")
    return int(r[0]), (None if r[1] == 0xFFFFFFFFFFFFFFFF else (int(r[1]) >> 32, int(r[1]) & 0xFFFFFFFF))


def selfcheck_encoder(kind, bounds, chunk=1 << 12, stream=None):
    """Mismatches between the kernels' E4M3 ("fp8") or E2M1 ("nvfp4") encoder
    and the step table `bounds` (see ss24_selfcheck_encoder) over every finite
    fp32 bit pattern; returns (count, first mismatching bit pattern or None)."""
    k = _FMT[kind] if isinstance(kind, str) else int(kind)
    b = torch.as_tensor(np.asarray(bounds, dtype=np.uint32).view(np.int32)).cuda()
    res = torch.tensor([0, -1], dtype=torch.int64, device="cuda")
    for h0 in range(0, 1 << 16, chunk):
        n = min(chunk, (1 << 16) - h0)
        _check(lib().ss24_selfcheck_encoder(k, _ptr(b), b.numel(), h0, n, _ptr(res), _stream(stream)),
               "ss24_selfcheck_encoder")
    r = res.cpu().numpy().view("uint64")
    return int(r[0]), (None if r[1] == 0xFFFFFFFFFFFFFFFF else int(r[1]))


def _convert(name, t_in, out_dtype, stream=None):
    out = torch.empty(t_in.shape, dtype=out_dtype, device=t_in.device)
    _check(getattr(lib(), name)(_ptr(t_in), _ptr(out), t_in.numel(), _stream(stream)), name)
    return out


def encode_e4m3(t, stream=None):
    return _convert("ss24_encode_e4m3", t.contiguous(), torch.uint8, stream)


def decode_e4m3(t, stream=None):
    return _convert("ss24_decode_e4m3", t.contiguous(), torch.float32, stream)


def encode_e2m1(t, stream=None):
    return _convert("ss24_encode_e2m1", t.contiguous(), torch.uint8, stream)


def decode_e2m1(t, stream=None):
    return _convert("ss24_decode_e2m1", t.contiguous(), torch.float32, stream)
