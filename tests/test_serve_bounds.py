"""What the serving operators may read and write, as far as the host decides it: the sizes that the binding passes on,
and arguments that would leave the arrays or let rows overwrite each other (CPU only)."""
import ctypes

import pytest
import torch

import adapter_gemv_gb300 as m
from adapter_gemv_gb300 import serve
from test_serve_abi import ATTN, CACHE, LOGITS, ROWS, L, made  # noqa: F401


@pytest.fixture
def host_tensors(monkeypatch):
    """The binding takes host tensors for device ones; nothing is called with them."""
    at = lambda t, what, dtype=None: 0 if t is None else t.data_ptr()  # noqa: E731
    monkeypatch.setattr(m, "_dev", at)
    monkeypatch.setattr(serve, "_dev", at)


def logits_call(tokens, n):
    x, i = torch.zeros(n, 40), torch.zeros(n, dtype=torch.int32)
    return m.LogitsAdjust(x, x, tokens=tokens, prompt_len=i, total_len=i).struct


@pytest.mark.parametrize("first", [0, 1, 100, 199, 200])
@pytest.mark.parametrize("rows", [1, 3])
def test_a_history_that_is_part_of_a_wider_matrix(L, host_tensors, rows, first):  # noqa: F811
    """Rows are as long as the view is wide, not as far apart as the matrix's."""
    wide = torch.zeros((rows, 200), dtype=torch.int32)
    s = logits_call(wide[:, first:], rows)
    assert s.tokens_len == 200 - first
    assert s.tokens_stride >= s.tokens_len
    if first < 200:
        end = (rows - 1) * s.tokens_stride + s.tokens_len  # behind the last id that may be read
        assert s.tokens + 4 * end == wide.data_ptr() + 4 * wide.numel()
    else:
        assert s.tokens_stride == 0


@pytest.mark.parametrize("kw", [dict(tokens_len=-1), dict(tokens_len=8), dict(tokens_stride=1 << 31),
                                dict(tokens_stride=0, tokens_len=1)])
def test_history_lengths_are_refused(L, kw):  # noqa: F811
    s = made(m.mlora_logits, LOGITS, kw)
    assert L.lora_logits_adjust(ctypes.byref(s), None, None) == m.ERR_SHAPE


@pytest.mark.parametrize("vocab", [2 ** 31 - 1, 2 ** 31 - 4096, 2 ** 31 - 65536])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_vocabularies_whose_last_slice_passes_31_bits_are_refused(L, vocab, dtype):  # noqa: F811
    s = made(m.mlora_logits, LOGITS, dict(vocab=vocab, dtype=dtype, ld=1 << 31, ldo=1 << 31, mask_stride=1 << 26))
    assert L.lora_logits_adjust(ctypes.byref(s), None, None) == m.ERR_SHAPE


def test_in_place_rows_of_another_distance_are_refused(L):  # noqa: F811
    """out = in with rows further apart: a row's output would lie over other rows' inputs."""
    c = made(m.mlora_kv_cache, CACHE, {})
    for kw in (dict(ldo=104), dict(ld=104)):
        assert L.lora_logits_adjust(ctypes.byref(made(m.mlora_logits, LOGITS, kw)), None, None) == m.ERR_SHAPE
    for kw in (dict(ldq_out=520), dict(ldq=520)):
        assert L.lora_kv_append(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_rows, ROWS, kw)), 1, None, None) == m.ERR_SHAPE
    for kw in (dict(ldo=520), dict(ldq=520)):
        assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_attn, ATTN, kw)), 1, None, None) == m.ERR_SHAPE


def test_a_negative_number_of_rows_per_request_is_refused(L):  # noqa: F811
    c, a = made(m.mlora_kv_cache, CACHE, {}), made(m.mlora_kv_attn, ATTN, dict(num_rows=0))
    assert L.lora_kv_attention_ex(ctypes.byref(c), ctypes.byref(a), 1, -1, None, None) == m.ERR_SHAPE
    for rows in (0, 1, 9, 2 ** 31 - 1):
        assert L.lora_kv_attention_ex(ctypes.byref(c), ctypes.byref(a), 1, rows, None, None) == 0
