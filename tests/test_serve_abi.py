"""The serving operators on the host: the binding's structures match the header's, host-detectable bad
arguments are refused with the documented codes before anything is launched, empty calls launch
nothing, and the binding checks its tensors (CPU only)."""
import ctypes
import os

import pytest
import torch

import adapter_gemv_gb300 as m
import serve_ref
from test_abi_layout import c_layout

F = 0x100000  # an aligned, device-looking address: validation only inspects it


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from adapter_gemv_gb300 import build
        build.build()
    return m.lib()


@pytest.mark.parametrize("struct", ["mlora_kv_batch", "mlora_kv_cache", "mlora_kv_rows", "mlora_kv_attn", "mlora_logits"])
def test_struct_layouts_match(tmp_path, struct):
    cls = getattr(m, struct)
    c = c_layout(tmp_path, struct, [f for f, _ in cls._fields_])
    for f, _ in cls._fields_:
        desc = getattr(cls, f)
        assert (desc.offset, desc.size) == c[f], f"{struct}.{f}"
    assert ctypes.sizeof(cls) == c["sizeof"][0]


def made(cls, base, kw):
    s = cls()
    for k, v in {**base, **kw}.items():
        setattr(s, k, v)
    return s


BATCH = dict(num_requests=4, num_rows=9, page_tokens=16, max_pages=8, num_pages=64, table_stride=8, new_tokens=F, kv_len=F,
             kv_len_out=F, page_table=F, free_ring=F, free_state=F, free_state_out=F, row_request=F, position=F,
             cache_slot=F, seg_offsets=F, seg_slot=F)
CACHE = dict(dtype=0, num_layers=2, num_kv_heads=4, head_dim=64, page_tokens=16, num_pages=32, k=F, v=F, page_stride=8192,
             layer_stride=4096, token_stride=256, head_stride=64)
ROWS = dict(num_rows=3, num_q_heads=8, cache_slot=F, position=F, k=F, v=F, q=F, q_out=F, ldk=256, ldv=256, ldq=512,
            ldq_out=512, rope_cos=F, rope_sin=F, rotary_dim=64, max_position=100)
ATTN = dict(num_rows=3, num_q_heads=8, q=F, out=F, ldq=512, ldo=512, position=F, page_table=F, table_stride=8,
            num_requests=3, max_pages=8, scale=0.125, workspace=F, workspace_bytes=1 << 40)
LOGITS = dict(num_rows=3, vocab=100, dtype=2, num_requests=3, logits=F, out=F, ld=100, ldo=100, tokens=F, tokens_stride=7,
              prompt_len=F, total_len=F, bias_offsets=F, bias_token=F, bias_value=F, num_bias=5, mask=F, mask_stride=4,
              mask_index=F, num_masks=1)


@pytest.mark.parametrize("kw, code", [
    (dict(num_requests=-1), m.ERR_SHAPE), (dict(num_requests=m.KV_MAX_REQUESTS + 1), m.ERR_SHAPE),
    (dict(num_rows=-1), m.ERR_SHAPE), (dict(page_tokens=0), m.ERR_SHAPE), (dict(num_pages=0), m.ERR_SHAPE),
    (dict(max_pages=-1), m.ERR_SHAPE), (dict(table_stride=7), m.ERR_SHAPE),
    (dict(max_pages=1 << 28, table_stride=1 << 28), m.ERR_SHAPE), (dict(free_ring=0), m.ERR_NULL),
    (dict(free_state=0), m.ERR_NULL), (dict(free_state_out=0), m.ERR_NULL), (dict(kv_len=0), m.ERR_NULL),
    (dict(new_tokens=0), m.ERR_NULL), (dict(kv_len_out=0), m.ERR_NULL), (dict(page_table=0), m.ERR_NULL),
    (dict(cache_slot=0), m.ERR_NULL), (dict(position=0), m.ERR_NULL), (dict(row_request=0), m.ERR_NULL),
    (dict(cache_slot=F + 4), m.ERR_ALIGN), (dict(kv_len=F + 2), m.ERR_ALIGN), (dict(seg_offsets=F + 1), m.ERR_ALIGN)])
def test_layout_refusals(L, kw, code):
    assert L.lora_kv_layout(ctypes.byref(made(m.mlora_kv_batch, BATCH, kw)), None, None) == code


CACHE_REFUSALS = [
    (dict(dtype=2), m.ERR_DTYPE), (dict(k=0), m.ERR_NULL), (dict(v=0), m.ERR_NULL), (dict(num_layers=0), m.ERR_SHAPE),
    (dict(num_kv_heads=0), m.ERR_SHAPE), (dict(head_dim=0), m.ERR_SHAPE), (dict(head_dim=264), m.ERR_SHAPE),
    (dict(page_tokens=0), m.ERR_SHAPE), (dict(num_pages=0), m.ERR_SHAPE), (dict(page_stride=-8), m.ERR_SHAPE),
    (dict(head_dim=60), m.ERR_ALIGN), (dict(token_stride=260), m.ERR_ALIGN), (dict(head_stride=4), m.ERR_ALIGN),
    (dict(k=F + 8), m.ERR_ALIGN), (dict(v=F + 2), m.ERR_ALIGN)]


@pytest.mark.parametrize("kw, code", CACHE_REFUSALS)
def test_cache_refusals(L, kw, code):
    c = made(m.mlora_kv_cache, CACHE, kw)
    assert L.lora_kv_append(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_rows, ROWS, {})), 0, None, None) == code
    assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_attn, ATTN, {})), 0, None, None) == code


@pytest.mark.parametrize("kw, code", [
    (dict(num_rows=-1), m.ERR_SHAPE), (dict(num_q_heads=-1), m.ERR_SHAPE), (dict(cache_slot=0), m.ERR_NULL),
    (dict(position=0), m.ERR_NULL), (dict(k=0), m.ERR_NULL), (dict(v=0), m.ERR_NULL), (dict(q=0), m.ERR_NULL),
    (dict(q_out=0), m.ERR_NULL), (dict(ldk=248), m.ERR_SHAPE), (dict(ldv=260), m.ERR_ALIGN), (dict(q=F + 8), m.ERR_ALIGN),
    (dict(ldq=504), m.ERR_SHAPE), (dict(rope_cos=0), m.ERR_NULL), (dict(rope_cos=0, rope_sin=0), m.ERR_NULL),
    (dict(rotary_dim=24), m.ERR_ALIGN), (dict(rotary_dim=80), m.ERR_SHAPE), (dict(max_position=0), m.ERR_SHAPE),
    (dict(rope_sin=F + 8), m.ERR_ALIGN), (dict(cache_slot=F + 4), m.ERR_ALIGN)])
def test_append_refusals(L, kw, code):
    c = made(m.mlora_kv_cache, CACHE, {})
    assert L.lora_kv_append(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_rows, ROWS, kw)), 1, None, None) == code


@pytest.mark.parametrize("kw, code", [
    (dict(num_rows=-1), m.ERR_SHAPE), (dict(num_requests=-1), m.ERR_SHAPE), (dict(window=-1), m.ERR_SHAPE),
    (dict(num_q_heads=0), m.ERR_SHAPE), (dict(num_q_heads=6), m.ERR_SHAPE), (dict(scale=float("nan")), m.ERR_SHAPE),
    (dict(table_stride=4), m.ERR_SHAPE), (dict(max_pages=1 << 28, table_stride=1 << 28), m.ERR_SHAPE),
    (dict(q=0), m.ERR_NULL), (dict(out=0), m.ERR_NULL), (dict(position=0), m.ERR_NULL), (dict(page_table=0), m.ERR_NULL),
    (dict(workspace=0), m.ERR_NULL), (dict(workspace=F + 8), m.ERR_ALIGN), (dict(workspace_bytes=15), m.ERR_WORKSPACE),
    (dict(ldq=516), m.ERR_ALIGN), (dict(ldo=504), m.ERR_SHAPE), (dict(out=F + 8), m.ERR_ALIGN), (dict(lse=F + 2), m.ERR_ALIGN)])
def test_attention_refusals(L, kw, code):
    c = made(m.mlora_kv_cache, CACHE, {})
    rc = L.lora_kv_attention(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_attn, ATTN, kw)), 1, None, None)
    assert rc == code and L.lora_error_string(rc) != L.lora_error_string(-99)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), m.ERR_DTYPE), (dict(num_rows=-1), m.ERR_SHAPE), (dict(vocab=0), m.ERR_SHAPE), (dict(logits=0), m.ERR_NULL),
    (dict(out=0), m.ERR_NULL), (dict(ld=99), m.ERR_SHAPE), (dict(ldo=99), m.ERR_SHAPE), (dict(tokens=0), m.ERR_NULL),
    (dict(prompt_len=0), m.ERR_NULL), (dict(total_len=0), m.ERR_NULL), (dict(bias_offsets=0), m.ERR_NULL),
    (dict(bias_value=0), m.ERR_NULL), (dict(num_bias=-1), m.ERR_SHAPE), (dict(mask=0), m.ERR_NULL),
    (dict(mask_index=0), m.ERR_NULL), (dict(num_masks=0), m.ERR_SHAPE), (dict(mask_stride=3), m.ERR_SHAPE),
    (dict(logits=F + 2), m.ERR_ALIGN), (dict(mask=F + 2), m.ERR_ALIGN), (dict(tokens_stride=-1), m.ERR_SHAPE)])
def test_logits_refusals(L, kw, code):
    assert L.lora_logits_adjust(ctypes.byref(made(m.mlora_logits, LOGITS, kw)), None, None) == code


def test_null_structs_and_layers(L):
    c, a, r = made(m.mlora_kv_cache, CACHE, {}), made(m.mlora_kv_attn, ATTN, {}), made(m.mlora_kv_rows, ROWS, {})
    assert L.lora_kv_layout(None, None, None) == m.ERR_NULL
    assert L.lora_kv_append(None, ctypes.byref(r), 0, None, None) == m.ERR_NULL
    assert L.lora_kv_append(ctypes.byref(c), None, 0, None, None) == m.ERR_NULL
    assert L.lora_kv_attention(None, ctypes.byref(a), 0, None, None) == m.ERR_NULL
    assert L.lora_logits_adjust(None, None, None) == m.ERR_NULL
    for layer in (-1, 2):
        assert L.lora_kv_append(ctypes.byref(c), ctypes.byref(r), layer, None, None) == m.ERR_SHAPE
        assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(a), layer, None, None) == m.ERR_SHAPE


def test_zero_rows_launch_nothing(L):
    before = L.lora_launch_count()
    c = made(m.mlora_kv_cache, CACHE, {})
    none = dict(num_rows=0, k=0, v=0, q=0, q_out=0, cache_slot=0, position=0)
    assert L.lora_kv_append(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_rows, ROWS, none)), 0, None, None) == 0
    none = dict(num_rows=0, q=0, out=0, position=0, workspace=0, workspace_bytes=0)
    assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(made(m.mlora_kv_attn, ATTN, none)), 0, None, None) == 0
    none = dict(num_rows=0, logits=0, out=0)
    assert L.lora_logits_adjust(ctypes.byref(made(m.mlora_logits, LOGITS, none)), None, None) == 0
    assert L.lora_launch_count() == before


def test_workspace_size(L):
    c = made(m.mlora_kv_cache, CACHE, {})
    n = L.lora_kv_attention_workspace(ctypes.byref(c), 8)
    assert n >= 0 and n % 16 == 0
    assert L.lora_kv_attention_workspace(None, 8) == 0


def test_binding_refuses_wrong_tensors():
    k = torch.zeros((1, 4, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.make_kv_cache(k, k.clone())
    with pytest.raises(ValueError, match="5-D"):
        m.make_kv_cache(k[0], k[0])
    with pytest.raises(ValueError, match="layout"):
        m.make_kv_cache(k, k.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(TypeError, match="bfloat16"):
        m.make_kv_cache(k.float(), k.float())
    with pytest.raises(ValueError, match="shape"):
        m.Rope(torch.zeros(4, 8), torch.zeros(4, 16))
    with pytest.raises(TypeError, match="float32"):
        m.LogitsAdjust(torch.zeros(1, 8).double(), torch.zeros(1, 8).double())
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        m.KvBatch(i, i, torch.zeros((2, 4), dtype=torch.int32), i, i, 16, 3)


def test_layout_reference_by_hand():
    """Two requests and a leaver, pages of 4: worked out by hand."""
    got = serve_ref.layout([3, -1, 1], [2, 5, 4], [[7, -1], [1, 0], [2, -1]], [9, 9, 9, 4, 3, 9, 9, 9], [3, 2], 4, 6,
                           [5, 6, 7])
    assert got["status"] == 0
    assert got["page_table"] == [[7, 4], [1, 0], [2, 3]]
    assert got["free_ring"] == [9, 9, 9, 4, 3, 1, 0, 9]
    assert got["free_state_out"] == [5, 2] and got["kv_len_out"] == [5, 0, 5]
    assert got["seg_offsets"] == [0, 3, 3, 4, 6] and got["seg_slot"] == [5, 6, 7, -1]
    assert got["row_request"] == [0, 0, 0, 2, -1, -1] and got["position"] == [2, 3, 4, 4, -1, -1]
    assert got["cache_slot"] == [30, 31, 16, 12, -1, -1] and got["row_slot"] == [5, 5, 5, 7, -1, -1]


def test_the_current_stream_with_and_without_torchs_private_call(monkeypatch):
    import types
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(m, "_raw_stream", lambda device: 1000 + device)
    assert m._stream(None) == 1003
    monkeypatch.setattr(m, "_raw_stream", None)
    assert m._stream(None) == 77
    assert m._stream(types.SimpleNamespace(cuda_stream=5)) == 5 and m._stream(9) == 9


def test_the_package_imports_without_torchs_private_call():
    import subprocess
    import sys
    code = ("import torch; hasattr(torch._C, '_cuda_getCurrentRawStream') and delattr(torch._C, '_cuda_getCurrentRawStream')\n"
            "import types; torch.cuda.current_stream = lambda: types.SimpleNamespace(cuda_stream=77)\n"
            "torch.cuda.current_device = lambda: 0\n"
            "import adapter_gemv_gb300 as m; assert m._stream(None) == 77")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
