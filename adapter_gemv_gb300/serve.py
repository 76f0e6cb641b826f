"""Binding of the operators around the adapted projections: the paged key-value cache's layout, the
write of new rows into it, the attention that reads it, and the per-request logit adjustment
(include/mlora.h, "the step around the adapters").

Argument marshalling only, like the package's other calls. A call's pointers and sizes are gathered
once in a prepared object (:class:`KvBatch`, :class:`KvAppend`, :class:`KvAttention`,
:class:`LogitsAdjust`) that a serving loop keeps with its buffers and calls for every step; the
functions named like the C entry points prepare and call in one go. Prepared objects hold references to
their tensors.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import MLORA_BF16, MLORA_FP16, SIGNATURES, _check, _dev, _i32, _rows, _stream, lib

MLORA_FP32 = 2
KV_MAX_REQUESTS = 8192
KV_MAX_HEAD_DIM = 256
STATUS_NO_PAGES, STATUS_BAD_LENGTH, STATUS_BAD_TOKEN, STATUS_BAD_REQUEST = 32, 64, 128, 256
ERR_WORKSPACE = -8

_DT = {torch.bfloat16: MLORA_BF16, torch.float16: MLORA_FP16}
_LOGIT_DT = {**_DT, torch.float32: MLORA_FP32}
_I, _L, _F, _V = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class mlora_kv_batch(ctypes.Structure):
    _fields_ = [("num_requests", _I), ("num_rows", _I), ("page_tokens", _I), ("max_pages", _I), ("num_pages", _I),
                ("table_stride", _L), ("new_tokens", _V), ("kv_len", _V), ("kv_len_out", _V), ("page_table", _V),
                ("free_ring", _V), ("free_state", _V), ("free_state_out", _V), ("adapter_slot", _V),
                ("row_request", _V), ("position", _V), ("cache_slot", _V), ("row_slot", _V), ("seg_offsets", _V),
                ("seg_slot", _V)]


class mlora_kv_cache(ctypes.Structure):
    _fields_ = [("dtype", _I), ("num_layers", _I), ("num_kv_heads", _I), ("head_dim", _I), ("page_tokens", _I),
                ("num_pages", _I), ("k", _V), ("v", _V), ("page_stride", _L), ("layer_stride", _L),
                ("token_stride", _L), ("head_stride", _L)]


class mlora_kv_rows(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("num_q_heads", _I), ("cache_slot", _V), ("position", _V), ("k", _V), ("v", _V),
                ("q", _V), ("q_out", _V), ("ldk", _L), ("ldv", _L), ("ldq", _L), ("ldq_out", _L), ("rope_cos", _V),
                ("rope_sin", _V), ("rotary_dim", _I), ("max_position", _I), ("rope_interleaved", _I)]


class mlora_kv_attn(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("num_q_heads", _I), ("q", _V), ("out", _V), ("ldq", _L), ("ldo", _L),
                ("position", _V), ("row_request", _V), ("page_table", _V), ("table_stride", _L), ("num_requests", _I),
                ("max_pages", _I), ("window", _I), ("scale", _F), ("lse", _V), ("workspace", _V),
                ("workspace_bytes", _L)]


class mlora_logits(ctypes.Structure):
    _fields_ = [("num_rows", _I), ("vocab", _I), ("dtype", _I), ("num_requests", _I), ("logits", _V), ("out", _V),
                ("ld", _L), ("ldo", _L), ("row_request", _V), ("tokens", _V), ("tokens_stride", _L), ("prompt_len", _V),
                ("total_len", _V), ("repetition", _V), ("presence", _V), ("frequency", _V), ("temperature", _V),
                ("bias_offsets", _V), ("bias_token", _V), ("bias_value", _V), ("num_bias", _I), ("mask", _V),
                ("mask_stride", _L), ("mask_index", _V), ("num_masks", _I), ("tokens_len", _I)]


_PC = ctypes.POINTER(mlora_kv_cache)
SIGNATURES.update({
    "lora_kv_layout": [ctypes.POINTER(mlora_kv_batch), _V, _V],
    "lora_kv_append": [_PC, ctypes.POINTER(mlora_kv_rows), _I, _V, _V],
    "lora_kv_attention": [_PC, ctypes.POINTER(mlora_kv_attn), _I, _V, _V],
    "lora_kv_attention_ex": [_PC, ctypes.POINTER(mlora_kv_attn), _I, _I, _V, _V],
    "lora_logits_adjust": [ctypes.POINTER(mlora_logits), _V, _V],
})


def _vec(t: Optional[torch.Tensor], what: str, n: int, dtype=torch.int32) -> int:
    """Pointer of a contiguous 1-D tensor of n entries (0 for None)."""
    if t is None:
        return 0
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-D tensor of {n} entries, got {tuple(t.shape)}")
    return _dev(t, what, dtype)


def _matrix(t: torch.Tensor, what: str, dtype, rows: int, cols: int) -> int:
    """Row stride of a 2-D tensor of at least rows x cols (the pointer is taken apart)."""
    ld = _rows(t, what, dtype)
    if t.shape[0] != rows or t.shape[1] < cols:
        raise ValueError(f"{what} must be [{rows}][>= {cols}], got {tuple(t.shape)}")
    return ld if rows > 1 else max(ld, t.shape[1])  # a single row's stride says nothing


class KvBatch:
    """A step's requests and rows (mlora_kv_batch): the tensors :func:`lora_kv_layout` reads and writes.

    new_tokens, kv_len: int32 [num_requests]; page_table: int32 [num_requests][max_pages]; free_ring:
    int32 [num_pages]; free_state: int32 [2] (head, count). kv_len_out and free_state_out default to
    kv_len and free_state, which each call then advances. The row arrays and the SGMV segments are
    allocated here, for num_rows rows, and written by every call.
    """

    def __init__(self, new_tokens, kv_len, page_table, free_ring, free_state, page_tokens: int, num_rows: int,
                 adapter_slot=None, kv_len_out=None, free_state_out=None):
        n, dev = int(kv_len.numel()), kv_len.device
        self.new_tokens, self.kv_len, self.page_table = new_tokens, kv_len, page_table
        self.free_ring, self.free_state, self.adapter_slot = free_ring, free_state, adapter_slot
        self.kv_len_out = kv_len if kv_len_out is None else kv_len_out
        self.free_state_out = free_state if free_state_out is None else free_state_out
        i32 = dict(dtype=torch.int32, device=dev)
        self.row_request, self.position = torch.empty(num_rows, **i32), torch.empty(num_rows, **i32)
        self.row_slot = torch.empty(num_rows, **i32)
        self.cache_slot = torch.empty(num_rows, dtype=torch.int64, device=dev)
        self.seg_offsets, self.seg_slot = torch.empty(n + 2, **i32), torch.empty(n + 1, **i32)
        s = self.struct = mlora_kv_batch()
        s.num_requests, s.num_rows, s.page_tokens = n, int(num_rows), int(page_tokens)
        s.max_pages, s.num_pages = int(page_table.shape[1]), int(free_ring.numel())
        s.table_stride = _matrix(page_table, "page_table", torch.int32, n, 0)
        s.new_tokens, s.kv_len = _vec(new_tokens, "new_tokens", n), _vec(kv_len, "kv_len", n)
        s.kv_len_out = _vec(self.kv_len_out, "kv_len_out", n)
        s.page_table = page_table.data_ptr()
        s.free_ring = _vec(free_ring, "free_ring", s.num_pages)
        s.free_state = _vec(free_state, "free_state", 2)
        s.free_state_out = _vec(self.free_state_out, "free_state_out", 2)
        s.adapter_slot = _vec(adapter_slot, "adapter_slot", n)
        s.row_request, s.position = self.row_request.data_ptr(), self.position.data_ptr()
        s.cache_slot, s.row_slot = self.cache_slot.data_ptr(), self.row_slot.data_ptr()
        s.seg_offsets, s.seg_slot = self.seg_offsets.data_ptr(), self.seg_slot.data_ptr()
        self.ref, self.fn = ctypes.pointer(s), lib().lora_kv_layout


def lora_kv_layout(batch: KvBatch, status=None, stream=None) -> None:
    """Pages and row places of a step from its requests' lengths (writes the batch's arrays)."""
    _check(batch.fn(batch.ref, 0 if status is None else _i32(status, "status"), _stream(stream)))


class KvCache:
    """A paged cache: k, v views [num_layers][num_pages][page_tokens][num_kv_heads][head_dim] with the
    same strides (any, multiples of 8 elements; head_dim unit-strided)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.stride(4) != 1:
            raise ValueError("k and v must be 5-D views of one shape and layout, the last dimension unit-strided")
        if k.dtype not in _DT:
            raise TypeError(f"the cache must be bfloat16 or float16, got {k.dtype}")
        self.k, self.v, self.dtype = k, v, k.dtype
        s = self.struct = mlora_kv_cache()
        s.dtype = _DT[k.dtype]
        s.num_layers, s.num_pages, s.page_tokens, s.num_kv_heads, s.head_dim = k.shape
        s.k, s.v = _dev(k, "k cache", k.dtype), _dev(v, "v cache", k.dtype)
        # the stride of a dimension of one entry says nothing
        s.layer_stride, s.page_stride, s.token_stride, s.head_stride = (
            st if n > 1 else 0 for st, n in zip(k.stride()[:4], k.shape[:4]))
        self.ref = ctypes.pointer(s)


def make_kv_cache(k, v=None) -> KvCache:
    return k if isinstance(k, KvCache) else KvCache(k, v)


class Rope:
    """Rotary tables cos, sin: fp32 [max_position][rotary_dim / 2]; pairs are (m, m + rotary_dim/2) of a
    head, or (2m, 2m + 1) with interleaved."""

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, interleaved: bool = False):
        if cos.dim() != 2 or cos.shape != sin.shape or not (cos.is_contiguous() and sin.is_contiguous()):
            raise ValueError("cos and sin must be contiguous 2-D tensors of one shape")
        _dev(cos, "cos", torch.float32), _dev(sin, "sin", torch.float32)
        self.cos, self.sin, self.interleaved = cos, sin, bool(interleaved)


class KvAppend:
    """A prepared lora_kv_append call."""

    def __init__(self, cache, k, v, cache_slot, layer: int, q=None, q_out=None, position=None,
                 rope: Optional[Rope] = None, status=None):
        c = self.cache = make_kv_cache(cache)
        n, dt = int(cache_slot.numel()), c.dtype
        d, hk = c.struct.head_dim, c.struct.num_kv_heads
        self.keep = (k, v, cache_slot, q, q_out, position, rope, status)
        s = self.struct = mlora_kv_rows()
        s.num_rows = n
        s.cache_slot = _vec(cache_slot, "cache_slot", n, torch.int64)
        s.position = _vec(position, "position", n)
        s.k, s.ldk = k.data_ptr(), _matrix(k, "k", dt, n, hk * d)
        s.v, s.ldv = v.data_ptr(), _matrix(v, "v", dt, n, hk * d)
        if q is not None:
            if q.shape[1] % d:
                raise ValueError("q must hold whole heads")
            s.num_q_heads = int(q.shape[1]) // d
            q_out = q if q_out is None else q_out
            s.q, s.ldq = q.data_ptr(), _matrix(q, "q", dt, n, q.shape[1])
            s.q_out, s.ldq_out = q_out.data_ptr(), _matrix(q_out, "q_out", dt, n, q.shape[1])
        if rope is not None:
            s.rope_cos, s.rope_sin = rope.cos.data_ptr(), rope.sin.data_ptr()
            s.max_position, s.rotary_dim = int(rope.cos.shape[0]), 2 * int(rope.cos.shape[1])
            s.rope_interleaved = int(rope.interleaved)
        self.ref, self.layer, self.status = ctypes.pointer(s), int(layer), _i32(status, "status")
        self.fn = lib().lora_kv_append

    def __call__(self, stream=None):
        _check(self.fn(self.cache.ref, self.ref, self.layer, self.status, _stream(stream)))


def lora_kv_append(cache, k, v, cache_slot, layer, q=None, q_out=None, position=None, rope=None, status=None,
                   stream=None) -> None:
    """Store rows k, v (columns: kv heads x head_dim) at their cache slots, k and q rotated by position
    where rope is given; q rotated into q_out (default: in place)."""
    KvAppend(cache, k, v, cache_slot, layer, q, q_out, position, rope, status)(stream)


def lora_kv_attention_workspace(cache, num_q_heads: int) -> int:
    """Bytes of workspace that lora_kv_attention needs on this cache, whatever the batch."""
    return int(lib().lora_kv_attention_workspace(make_kv_cache(cache).ref, int(num_q_heads)))


def kv_attention_workspace(cache, num_q_heads: int) -> torch.Tensor:
    """A workspace for lora_kv_attention on this cache: zeroed once, kept for every call on one stream."""
    c = make_kv_cache(cache)
    return torch.zeros(lora_kv_attention_workspace(c, num_q_heads), dtype=torch.uint8, device=c.k.device)


class KvAttention:
    """A prepared lora_kv_attention call. Row i of q and out is a token of request row_request[i] (default:
    request i) that sees the cached tokens 0 .. position[i], the last `window` of them if window > 0. rows_per_request: how
    many rows a request has at most (1: a decode step), 0 if that is not known; it decides the time only."""

    def __init__(self, out, q, cache, page_table, position, layer: int, workspace, row_request=None, lse=None,
                 scale: Optional[float] = None, window: int = 0, status=None, rows_per_request: int = 0):
        c = self.cache = make_kv_cache(cache)
        n, d = int(position.numel()), c.struct.head_dim
        if q.shape[1] % d:
            raise ValueError("q must hold whole heads")
        hq = int(q.shape[1]) // d
        self.keep = (out, q, page_table, position, workspace, row_request, lse, status)
        s = self.struct = mlora_kv_attn()
        s.num_rows, s.num_q_heads = n, hq
        s.q, s.ldq = q.data_ptr(), _matrix(q, "q", c.dtype, n, hq * d)
        s.out, s.ldo = out.data_ptr(), _matrix(out, "out", c.dtype, n, hq * d)
        s.position, s.row_request = _vec(position, "position", n), _vec(row_request, "row_request", n)
        s.page_table = page_table.data_ptr()
        s.num_requests, s.max_pages = (int(x) for x in page_table.shape)
        s.table_stride = _matrix(page_table, "page_table", torch.int32, s.num_requests, 0)
        s.scale, s.window = d ** -0.5 if scale is None else float(scale), int(window)
        if lse is not None:
            if tuple(lse.shape) != (n, hq) or not lse.is_contiguous():
                raise ValueError(f"lse must be contiguous [{n}][{hq}]")
            s.lse = _dev(lse, "lse", torch.float32)
        s.workspace, s.workspace_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
        self.ref, self.layer, self.status = ctypes.pointer(s), int(layer), _i32(status, "status")
        self.fn, self.rows_per_request = lib().lora_kv_attention_ex, int(rows_per_request)

    def __call__(self, stream=None):
        _check(self.fn(self.cache.ref, self.ref, self.layer, self.rows_per_request, self.status, _stream(stream)))


def lora_kv_attention(out, q, cache, page_table, position, layer, workspace, row_request=None, lse=None, scale=None,
                      window=0, status=None, stream=None) -> None:
    """Attention of rows q (columns: query heads x head_dim) over the paged cache, into out."""
    KvAttention(out, q, cache, page_table, position, layer, workspace, row_request, lse, scale, window, status)(stream)


def lora_kv_attention_ex(out, q, cache, page_table, position, layer, workspace, rows_per_request, row_request=None,
                         lse=None, scale=None, window=0, status=None, stream=None) -> None:
    """The same, told how many rows a request has at most."""
    KvAttention(out, q, cache, page_table, position, layer, workspace, row_request, lse, scale, window, status,
                rows_per_request)(stream)


class LogitsAdjust:
    """A prepared lora_logits_adjust call. Per-request arrays (num_requests entries) are indexed by
    row_request (default: row i is request i); bias is (offsets, token, value), a list per request."""

    def __init__(self, out, logits, row_request=None, tokens=None, prompt_len=None, total_len=None, repetition=None,
                 presence=None, frequency=None, temperature=None,
                 bias: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None, mask=None, mask_index=None,
                 status=None):
        if logits.dtype not in _LOGIT_DT:
            raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
        rows, vocab = (int(x) for x in logits.shape)
        self.keep = (out, logits, row_request, tokens, prompt_len, total_len, repetition, presence, frequency,
                     temperature, bias, mask, mask_index, status)
        lists = [t for t in (total_len, prompt_len, repetition, presence, frequency, temperature, mask_index)
                 if t is not None]
        n = int(lists[0].numel()) if lists else int(bias[0].numel()) - 1 if bias is not None else rows
        if row_request is None and n < rows:
            raise ValueError(f"{rows} rows for {n} requests: give row_request")
        s = self.struct = mlora_logits()
        s.num_rows, s.vocab, s.dtype, s.num_requests = rows, vocab, _LOGIT_DT[logits.dtype], n
        s.logits, s.ld = logits.data_ptr(), _matrix(logits, "logits", logits.dtype, rows, vocab)
        s.out, s.ldo = out.data_ptr(), _matrix(out, "out", logits.dtype, rows, vocab)
        s.row_request = _vec(row_request, "row_request", rows)
        if tokens is not None:
            s.tokens = tokens.data_ptr()
            s.tokens_stride, s.tokens_len = _matrix(tokens, "tokens", torch.int32, n, 0), int(tokens.shape[1])
            if not s.tokens_len:
                s.tokens_stride = 0  # (a length of 0 alone would mean the stride)
        s.prompt_len, s.total_len = _vec(prompt_len, "prompt_len", n), _vec(total_len, "total_len", n)
        for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency),
                        ("temperature", temperature)):
            setattr(s, name, _vec(t, name, n, torch.float32))
        if bias is not None:
            off, tok, val = bias
            s.num_bias = int(tok.numel())
            s.bias_offsets = _vec(off, "bias offsets", n + 1)
            s.bias_token = _vec(tok, "bias tokens", s.num_bias)
            s.bias_value = _vec(val, "bias values", s.num_bias, torch.float32)
        if mask is not None:
            s.mask, s.num_masks = mask.data_ptr(), int(mask.shape[0])
            s.mask_stride = _matrix(mask, "mask", torch.int32, s.num_masks, (vocab + 31) // 32)
        s.mask_index = _vec(mask_index, "mask_index", n)
        self.ref, self.status = ctypes.pointer(s), _i32(status, "status")
        self.fn = lib().lora_logits_adjust

    def __call__(self, stream=None):
        _check(self.fn(self.ref, self.status, _stream(stream)))


def lora_logits_adjust(out, logits, row_request=None, tokens=None, prompt_len=None, total_len=None, repetition=None,
                       presence=None, frequency=None, temperature=None, bias=None, mask=None, mask_index=None,
                       status=None, stream=None) -> None:
    """Penalties, biases, temperature and grammar mask (int32 words of 32 bits) of each request's logits."""
    LogitsAdjust(out, logits, row_request, tokens, prompt_len, total_len, repetition, presence, frequency, temperature,
                 bias, mask, mask_index, status)(stream)
