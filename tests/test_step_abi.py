"""The norm, 8-bit rows, base product and sampling on the host: the binding's structures match the header's, host-detectable bad
arguments are refused with the documented codes before anything is launched, empty calls launch nothing, and
the binding checks its tensors (CPU only)."""
import ctypes

import pytest
import torch

import adapter_gemv_gb300 as m
from adapter_gemv_gb300 import step
from test_abi_layout import c_layout
from test_serve_abi import F, L, made  # noqa: F401
from test_serve_bounds import host_tensors  # noqa: F401

G, H = F + (1 << 20), F + (2 << 20)
NORM = dict(num_rows=3, width=264, dtype=0, eps=1e-5, x=F, residual=G, weight=F, residual_out=G, out=H, q=H + 4096, q_scale=F, ldx=264,
            ldr=264, ldro=264, ldo=264, ldq=264, lds=3)
QUANT = dict(num_rows=3, width=264, dtype=1, x=F, gate=G, out=H, q=H + 4096, q_scale=F, ldx=264, ldg=264, ldo=264, ldq=264, lds=3)
MATMUL = dict(num_rows=3, d_in=272, d_out=136, dtype=0, x=F, x_scale=F, w=G, w_scale=G, y=H, ldx=272, ldxs=3, ldw=272, ldws=3, ldy=136)
SAMPLING = dict(num_rows=3, vocab=1001, dtype=2, num_requests=3, logits=F, ld=1001, uniform=F, temperature=F, top_k=F, top_p=F, min_p=F,
                token=G, logprob=G)


@pytest.mark.parametrize("struct", ["mlora_norm", "mlora_quant", "mlora_matmul", "mlora_sampling"])
def test_struct_layouts_match(tmp_path, struct):
    cls = getattr(m, struct)
    c = c_layout(tmp_path, struct, [f for f, _ in cls._fields_])
    for f, _ in cls._fields_:
        desc = getattr(cls, f)
        assert (desc.offset, desc.size) == c[f], f"{struct}.{f}"
    assert ctypes.sizeof(cls) == c["sizeof"][0]


def call(L, name, kw, base):  # noqa: F811
    cls, fn = {"norm": (m.mlora_norm, L.lora_rms_norm), "quant": (m.mlora_quant, L.lora_quantize),
               "matmul": (m.mlora_matmul, L.lora_fp8_matmul), "sampling": (m.mlora_sampling, L.lora_sample)}[name]
    a = ctypes.byref(made(cls, base, kw))
    return fn(a, None, None) if name in ("matmul", "sampling") else fn(a, None)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=2), m.ERR_DTYPE), (dict(num_rows=-1), m.ERR_SHAPE), (dict(width=0), m.ERR_SHAPE), (dict(width=m.ROW_MAX_WIDTH + 8), m.ERR_SHAPE),
    (dict(width=260), m.ERR_ALIGN), (dict(eps=0.0), m.ERR_SHAPE), (dict(eps=-1.0), m.ERR_SHAPE), (dict(eps=float("nan")), m.ERR_SHAPE),
    (dict(eps=float("inf")), m.ERR_SHAPE), (dict(x=0), m.ERR_NULL), (dict(residual=0), m.ERR_NULL), (dict(residual_out=0), m.ERR_NULL),
    (dict(out=0, q=0, q_scale=0), m.ERR_NULL), (dict(q=0), m.ERR_NULL), (dict(q_scale=0), m.ERR_NULL), (dict(x=F + 8), m.ERR_ALIGN),
    (dict(weight=F + 2), m.ERR_ALIGN), (dict(q=H + 4104), m.ERR_ALIGN), (dict(q_scale=F + 2), m.ERR_ALIGN), (dict(ldx=256), m.ERR_SHAPE),
    (dict(ldr=268), m.ERR_ALIGN), (dict(ldo=256), m.ERR_SHAPE), (dict(ldq=268), m.ERR_ALIGN), (dict(lds=2), m.ERR_SHAPE),
    (dict(ldro=272), m.ERR_SHAPE), (dict(out=F, ldo=272), m.ERR_SHAPE), (dict(out=G), m.ERR_SHAPE), (dict(residual_out=H), m.ERR_SHAPE),
    (dict(residual_out=F, ldro=272), m.ERR_SHAPE), (dict(q=H), m.ERR_SHAPE), (dict(q=G), m.ERR_SHAPE)])
def test_norm_refusals(L, kw, code):  # noqa: F811
    assert call(L, "norm", kw, NORM) == code


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=2), m.ERR_DTYPE), (dict(num_rows=-1), m.ERR_SHAPE), (dict(width=0), m.ERR_SHAPE), (dict(width=2 ** 31 - 8), m.ERR_SHAPE),
    (dict(width=260), m.ERR_ALIGN), (dict(x=0), m.ERR_NULL), (dict(out=0, q=0, q_scale=0), m.ERR_NULL), (dict(q=0), m.ERR_NULL),
    (dict(q_scale=0), m.ERR_NULL), (dict(gate=G + 8), m.ERR_ALIGN), (dict(ldg=256), m.ERR_SHAPE), (dict(ldo=268), m.ERR_ALIGN),
    (dict(ldq=256), m.ERR_SHAPE), (dict(lds=2), m.ERR_SHAPE), (dict(out=F, ldo=272), m.ERR_SHAPE), (dict(out=G, ldo=272), m.ERR_SHAPE),
    (dict(q=H), m.ERR_SHAPE)])
def test_quantize_refusals(L, kw, code):  # noqa: F811
    assert call(L, "quant", kw, QUANT) == code


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=2), m.ERR_DTYPE), (dict(num_rows=-1), m.ERR_SHAPE), (dict(d_in=0), m.ERR_SHAPE), (dict(d_out=0), m.ERR_SHAPE),
    (dict(d_out=2 ** 31 - 128, ldy=2 ** 31), m.ERR_SHAPE), (dict(d_in=264), m.ERR_ALIGN), (dict(d_out=132), m.ERR_ALIGN), (dict(x=0), m.ERR_NULL), (dict(w=0), m.ERR_NULL), (dict(y=0), m.ERR_NULL),
    (dict(x_scale=0), m.ERR_NULL), (dict(w_scale=0), m.ERR_NULL), (dict(x=F + 8), m.ERR_ALIGN), (dict(w=G + 4), m.ERR_ALIGN),
    (dict(y=H + 8), m.ERR_ALIGN), (dict(x_scale=F + 2), m.ERR_ALIGN), (dict(ldx=256), m.ERR_SHAPE), (dict(ldx=280), m.ERR_ALIGN),
    (dict(ldw=280), m.ERR_ALIGN), (dict(ldw=256), m.ERR_SHAPE), (dict(ldxs=2), m.ERR_SHAPE), (dict(ldws=2), m.ERR_SHAPE),
    (dict(ldy=128), m.ERR_SHAPE), (dict(ldy=140), m.ERR_ALIGN), (dict(y=F), m.ERR_SHAPE), (dict(y=G), m.ERR_SHAPE)])
def test_matmul_refusals(L, kw, code):  # noqa: F811
    assert call(L, "matmul", kw, MATMUL) == code


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), m.ERR_DTYPE), (dict(num_rows=-1), m.ERR_SHAPE), (dict(vocab=0), m.ERR_SHAPE), (dict(num_requests=-1), m.ERR_SHAPE),
    (dict(vocab=m.SAMPLE_MAX_VOCAB + 1, ld=1 << 20), m.ERR_SHAPE), (dict(ld=1000), m.ERR_SHAPE), (dict(logits=0), m.ERR_NULL),
    (dict(uniform=0), m.ERR_NULL), (dict(token=0), m.ERR_NULL), (dict(logits=F + 2), m.ERR_ALIGN), (dict(dtype=0, logits=F + 1), m.ERR_ALIGN),
    (dict(top_k=F + 2), m.ERR_ALIGN), (dict(token=G + 1), m.ERR_ALIGN), (dict(logprob=G + 2), m.ERR_ALIGN)])
def test_sample_refusals(L, kw, code):  # noqa: F811
    assert call(L, "sampling", kw, SAMPLING) == code


def test_null_structs_and_no_rows(L):  # noqa: F811
    assert L.lora_rms_norm(None, None) == L.lora_quantize(None, None) == m.ERR_NULL
    assert L.lora_fp8_matmul(None, None, None) == L.lora_sample(None, None, None) == m.ERR_NULL
    before = L.lora_launch_count()
    for name, base in (("norm", NORM), ("quant", QUANT), ("matmul", MATMUL), ("sampling", SAMPLING)):
        none = {k: 0 for k in base if k in ("x", "w", "y", "logits", "token", "uniform", "out", "q", "q_scale", "num_rows")}
        assert call(L, name, none, base) == 0
    assert L.lora_launch_count() == before


def test_binding_refuses_wrong_tensors(host_tensors, monkeypatch):  # noqa: F811
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256)).to(torch.float8_e4m3fn), torch.zeros((4, 2))
    with pytest.raises(TypeError, match="bfloat16"):
        m.RmsNorm(x.float(), out=x.float())
    with pytest.raises(ValueError, match="2-D"):
        m.Quantize(x[0], q, s)
    with pytest.raises(ValueError, match="out must be"):
        m.RmsNorm(x, out=torch.zeros((4, 248), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="q_scale must be"):
        m.Quantize(x, q, torch.zeros((4, 3)))
    with pytest.raises(ValueError, match="residual must be"):
        m.RmsNorm(x, residual=x[:3], out=x)
    with pytest.raises(ValueError, match="w_scale must be"):
        m.Fp8Matmul(x[:, :128], q, s, torch.zeros((128, 256)).to(torch.float8_e4m3fn), torch.zeros((2, 2)))
    with pytest.raises(ValueError, match="give row_request"):
        m.Sample(torch.zeros(4, dtype=torch.int32), x, torch.zeros(4), temperature=torch.ones(3))
    with pytest.raises(TypeError, match="logits"):
        m.Sample(torch.zeros(4, dtype=torch.int32), x.double(), torch.zeros(4))
    monkeypatch.undo()
    with pytest.raises(ValueError, match="CUDA"):
        m.RmsNorm(x, out=x)
    with pytest.raises(TypeError, match="float8"):
        monkeypatch.setattr(torch.Tensor, "is_cuda", True)
        m.Quantize(x, x.to(torch.float16), s)


def test_a_single_rows_stride_says_nothing(L, host_tensors):  # noqa: F811
    wide = torch.zeros((1, 3, 264), dtype=torch.bfloat16)[:, 0]
    c = m.Quantize(wide, out=torch.zeros((1, 264), dtype=torch.bfloat16))
    assert c.struct.ldx >= 264 and c.struct.width == 264
    assert m.RmsNorm(wide, residual=wide, out=torch.zeros_like(wide)).struct.residual_out == wide.data_ptr()


def test_sizes_of_the_header_and_the_binding():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mlora.h")).read()
    for name, value in (("MLORA_FP8_BLOCK", step.FP8_BLOCK), ("MLORA_ROW_MAX_WIDTH", step.ROW_MAX_WIDTH),
                        ("MLORA_SAMPLE_MAX_VOCAB", step.SAMPLE_MAX_VOCAB)):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == value


def test_requests_without_limits_have_any_number(host_tensors):  # noqa: F811
    """A row of request 5 in a call of one row: no array of the requests that it could be outside of."""
    x, token, one = torch.zeros(1, 16), torch.zeros(1, dtype=torch.int32), torch.zeros(1)
    request = torch.tensor([5], dtype=torch.int32)
    assert m.Sample(token, x, one, row_request=request).struct.num_requests > 5
    assert m.Sample(token, x, one, row_request=request, temperature=torch.ones(3)).struct.num_requests == 3
    assert m.Sample(token, x, one).struct.num_requests == 1
