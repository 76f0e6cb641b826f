"""Binding of the operators between a step's adapted projections whose base weights are held in 8 bits: the
norm with the residual's addition, the 8-bit rows, the base product, and the choice of the next token
(include/mlora.h, "norm, 8-bit rows, base product, next token").

Argument marshalling only. As in :mod:`.serve`, a call's pointers and sizes are gathered once in a prepared object
(:class:`RmsNorm`, :class:`Quantize`, :class:`Fp8Matmul`, :class:`Sample`) that a serving loop keeps with its
buffers; the functions named like the C entry points prepare and call in one go. 8-bit rows are a
torch.float8_e4m3fn tensor [rows][width] and an fp32 tensor [rows][ceil(width / 128)] of their blocks' scales.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import SIGNATURES, _check, _i32, _stream, lib
from .serve import _DT, _LOGIT_DT, _matrix, _vec

FP8_BLOCK = 128
ROW_MAX_WIDTH = 32768
SAMPLE_MAX_VOCAB = 393216

_I, _L, _F, _V = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class mlora_norm(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("width", _I), ("dtype", _I), ("eps", _F), ("x", _V), ("residual", _V), ("weight", _V),
                ("residual_out", _V), ("out", _V), ("q", _V), ("q_scale", _V), ("ldx", _L), ("ldr", _L), ("ldro", _L),
                ("ldo", _L), ("ldq", _L), ("lds", _L)]


class mlora_quant(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("width", _I), ("dtype", _I), ("x", _V), ("gate", _V), ("out", _V), ("q", _V),
                ("q_scale", _V), ("ldx", _L), ("ldg", _L), ("ldo", _L), ("ldq", _L), ("lds", _L)]


class mlora_matmul(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("d_in", _I), ("d_out", _I), ("dtype", _I), ("x", _V), ("x_scale", _V), ("w", _V),
                ("w_scale", _V), ("y", _V), ("ldx", _L), ("ldxs", _L), ("ldw", _L), ("ldws", _L), ("ldy", _L)]


class mlora_sampling(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("vocab", _I), ("dtype", _I), ("num_requests", _I), ("logits", _V), ("ld", _L),
                ("row_request", _V), ("uniform", _V), ("temperature", _V), ("top_k", _V), ("top_p", _V), ("min_p", _V),
                ("token", _V), ("logprob", _V)]


SIGNATURES.update({
    "lora_rms_norm": [ctypes.POINTER(mlora_norm), _V],
    "lora_quantize": [ctypes.POINTER(mlora_quant), _V],
    "lora_fp8_matmul": [ctypes.POINTER(mlora_matmul), _V, _V],
    "lora_sample": [ctypes.POINTER(mlora_sampling), _V, _V],
})


def _type(x: torch.Tensor, what: str):
    if x.dtype not in _DT:
        raise TypeError(f"{what} must be bfloat16 or float16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor, got {tuple(x.shape)}")
    return x.dtype


def _blocks(columns: int) -> int:
    return (columns + FP8_BLOCK - 1) // FP8_BLOCK


def _optional(s, name: str, ld: str, t: Optional[torch.Tensor], dtype, rows: int, cols: int) -> None:
    """Pointer and row stride of a [rows][cols] tensor into the fields `name` and `ld`; None: neither."""
    if t is not None:
        if t.dim() == 2 and t.shape[1] != cols:
            raise ValueError(f"{name} must be [{rows}][{cols}], got {tuple(t.shape)}")
        setattr(s, ld, _matrix(t, name, dtype, rows, cols))
        setattr(s, name, t.data_ptr())


class _Call:
    def __call__(self, stream=None):
        _check(self.fn(self.ref, _stream(stream)))


class RmsNorm(_Call):
    """A prepared lora_rms_norm call: residual_out = x + residual, out and (q, q_scale) = its norm times weight. residual_out
    defaults to residual (in place); without a residual there is none."""

    def __init__(self, x, weight=None, eps: float = 1e-5, residual=None, residual_out=None, out=None, q=None, q_scale=None):
        dt = _type(x, "x")
        n, d = (int(i) for i in x.shape)
        if residual is not None and residual_out is None:
            residual_out = residual
        self.keep = (x, weight, residual, residual_out, out, q, q_scale)
        s = self.struct = mlora_norm()
        s.num_rows, s.width, s.dtype, s.eps = n, d, _DT[dt], float(eps)
        _optional(s, "x", "ldx", x, dt, n, d)
        _optional(s, "residual", "ldr", residual, dt, n, d)
        _optional(s, "residual_out", "ldro", residual_out, dt, n, d)
        _optional(s, "out", "ldo", out, dt, n, d)
        _optional(s, "q", "ldq", q, torch.float8_e4m3fn, n, d)
        _optional(s, "q_scale", "lds", q_scale, torch.float32, n, _blocks(d))
        s.weight = _vec(weight, "weight", d, dt)
        self.ref, self.fn = ctypes.pointer(s), lib().lora_rms_norm


def lora_rms_norm(x, weight=None, eps=1e-5, residual=None, residual_out=None, out=None, q=None, q_scale=None,
                  stream=None) -> None:
    """The residual's sum, its root-mean-square norm in 16 bits (out) and as 8-bit rows (q, q_scale)."""
    RmsNorm(x, weight, eps, residual, residual_out, out, q, q_scale)(stream)


class Quantize(_Call):
    """A prepared lora_quantize call: x, or silu(gate) * x, as 8-bit rows (q, q_scale) and in 16 bits (out)."""

    def __init__(self, x, q=None, q_scale=None, gate=None, out=None):
        dt = _type(x, "x")
        n, d = (int(i) for i in x.shape)
        self.keep = (x, q, q_scale, gate, out)
        s = self.struct = mlora_quant()
        s.num_rows, s.width, s.dtype = n, d, _DT[dt]
        _optional(s, "x", "ldx", x, dt, n, d)
        _optional(s, "gate", "ldg", gate, dt, n, d)
        _optional(s, "out", "ldo", out, dt, n, d)
        _optional(s, "q", "ldq", q, torch.float8_e4m3fn, n, d)
        _optional(s, "q_scale", "lds", q_scale, torch.float32, n, _blocks(d))
        self.ref, self.fn = ctypes.pointer(s), lib().lora_quantize


def lora_quantize(x, q=None, q_scale=None, gate=None, out=None, stream=None) -> None:
    """x, or silu(gate) * x, as 8-bit rows (q, q_scale) and in 16 bits (out)."""
    Quantize(x, q, q_scale, gate, out)(stream)


class _StatusCall(_Call):
    def __call__(self, stream=None):
        _check(self.fn(self.ref, self.status, _stream(stream)))


class Fp8Matmul(_StatusCall):
    """A prepared lora_fp8_matmul call: y [rows][d_out] = x w^T of 8-bit rows x, x_scale and weights w [d_out][d_in]
    with w_scale [ceil(d_out / 128)][ceil(d_in / 128)]."""

    def __init__(self, y, x, x_scale, w, w_scale, status=None):
        dt = _type(y, "y")
        if x.dim() != 2 or w.dim() != 2:
            raise ValueError(f"x and w must be 2-D tensors, got {tuple(x.shape)} and {tuple(w.shape)}")
        (n, k), m = (int(i) for i in x.shape), int(w.shape[0])
        self.keep = (y, x, x_scale, w, w_scale, status)
        s = self.struct = mlora_matmul()
        s.num_rows, s.d_in, s.d_out, s.dtype = n, k, m, _DT[dt]
        _optional(s, "x", "ldx", x, torch.float8_e4m3fn, n, k)
        _optional(s, "x_scale", "ldxs", x_scale, torch.float32, n, _blocks(k))
        _optional(s, "w", "ldw", w, torch.float8_e4m3fn, m, k)
        _optional(s, "w_scale", "ldws", w_scale, torch.float32, _blocks(m), _blocks(k))
        _optional(s, "y", "ldy", y, dt, n, m)
        self.ref, self.status, self.fn = ctypes.pointer(s), _i32(status, "status"), lib().lora_fp8_matmul


def lora_fp8_matmul(y, x, x_scale, w, w_scale, status=None, stream=None) -> None:
    """y = x w^T of 8-bit rows and 8-bit weights with a scale for each block of 128 x 128."""
    Fp8Matmul(y, x, x_scale, w, w_scale, status)(stream)


class Sample(_StatusCall):
    """A prepared lora_sample call: the next token of each row of logits from its random number in `uniform`. Per-request
    arrays are indexed by row_request (default: row i is request i)."""

    def __init__(self, token, logits, uniform, row_request=None, temperature=None, top_k=None, top_p=None, min_p=None,
                 logprob=None, status=None):
        if logits.dtype not in _LOGIT_DT:
            raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
        rows, vocab = (int(i) for i in logits.shape)
        self.keep = (token, logits, uniform, row_request, temperature, top_k, top_p, min_p, logprob, status)
        lists = [t for t in (temperature, top_k, top_p, min_p) if t is not None]
        # (without such arrays a request has nothing that its number could miss)
        n = int(lists[0].numel()) if lists else rows if row_request is None else 2 ** 31 - 1
        if row_request is None and n < rows:
            raise ValueError(f"{rows} rows for {n} requests: give row_request")
        s = self.struct = mlora_sampling()
        s.num_rows, s.vocab, s.dtype, s.num_requests = rows, vocab, _LOGIT_DT[logits.dtype], n
        s.logits, s.ld = logits.data_ptr(), _matrix(logits, "logits", logits.dtype, rows, vocab)
        s.row_request, s.token = _vec(row_request, "row_request", rows), _vec(token, "token", rows)
        s.uniform, s.logprob = _vec(uniform, "uniform", rows, torch.float32), _vec(logprob, "logprob", rows, torch.float32)
        s.temperature, s.top_k = _vec(temperature, "temperature", n, torch.float32), _vec(top_k, "top_k", n)
        s.top_p, s.min_p = _vec(top_p, "top_p", n, torch.float32), _vec(min_p, "min_p", n, torch.float32)
        self.ref, self.status, self.fn = ctypes.pointer(s), _i32(status, "status"), lib().lora_sample


def lora_sample(token, logits, uniform, row_request=None, temperature=None, top_k=None, top_p=None, min_p=None,
                logprob=None, status=None, stream=None) -> None:
    """The next token of each row from its random number, with temperature, top-k, top-p and min-p of its request."""
    Sample(token, logits, uniform, row_request, temperature, top_k, top_p, min_p, logprob, status)(stream)
