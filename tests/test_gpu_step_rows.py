"""lora_rms_norm and lora_quantize against their definitions in 64 bits (step_ref)."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import os
    if not os.path.exists(m.LIB_PATH):
        from adapter_gemv_gb300 import build
        build.build()
    return torch.device("cuda:0")


def normal(shape, dtype, dev, seed, std=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.empty(shape, device=dev).normal_(0, std, generator=g).to(dtype)


def framed(rows, cols, dtype, dev, pad=0, fill=77.0):
    """A [rows][cols] view of a wider array, and the array (its other columns stay as they are)."""
    wide = torch.full((rows, cols + pad), fill, device=dev).to(dtype)
    return wide[:, :cols], wide


def untouched(wide, cols, fill=77.0):
    return bool((wide[:, cols:].float() == torch.tensor(fill).to(wide.dtype).float().item()).all())


@pytest.mark.parametrize("rows, width", [(1, 8), (1, 128), (3, 120), (2, 136), (5, 2744), (33, 4096), (7, 8192), (4, 8200), (3, 11008),
                                         (2, 16392), (2, 32768), (1300, 520)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(dev, rows, width, dtype, with_residual):
    x, w = normal((rows, width), dtype, dev, 1), normal((width,), dtype, dev, 2, 0.3) + 1
    res = normal((rows, width), dtype, dev, 3, 3.0) if with_residual else None
    res_out, res_wide = framed(rows, width, dtype, dev, 8)
    out, out_wide = framed(rows, width, dtype, dev, 16)
    q, q_wide = framed(rows, width, ref.E4M3, dev, 24)
    scale, scale_wide = framed(rows, -(-width // 128), torch.float32, dev, 3)
    m.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=res_out if with_residual else None, out=out, q=q, q_scale=scale)
    h, v, rel = ref.norm(x, res, w, 1e-5)
    ref.within(out, v, rel, "out")
    ref.check_rows8(q, scale, v, rel, "q")
    assert untouched(out_wide, width) and untouched(q_wide, width) and untouched(scale_wide, scale.shape[1])
    if with_residual:
        ref.within(res_out, h, ref.U, "residual")
        assert untouched(res_wide, width)
    else:
        assert untouched(res_wide, 0)
    # each output alone: the same bits
    for kw in (dict(out=torch.empty_like(x)), dict(q=torch.empty_like(x, dtype=ref.E4M3), q_scale=torch.empty_like(scale))):
        m.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=torch.empty_like(x) if with_residual else None, **kw)
        for got, want in (("out", out), ("q", q), ("q_scale", scale)):
            if got in kw:
                assert torch.equal(kw[got].float(), want.float())


def test_norm_in_place_and_without_weight(dev):
    x, res = normal((37, 1000), BF16, dev, 1), normal((37, 1000), BF16, dev, 2)
    out, sums = torch.empty_like(x), torch.empty_like(x)
    m.lora_rms_norm(x, None, 1e-6, residual=res, residual_out=sums, out=out)
    a, b = x.clone(), res.clone()
    m.lora_rms_norm(a, None, 1e-6, residual=b, out=a)  # residual_out: the residual
    assert torch.equal(a, out) and torch.equal(b, sums)
    a, b = x.clone(), res.clone()
    m.lora_rms_norm(a, None, 1e-6, residual=b, residual_out=a, out=b)
    assert torch.equal(a, sums) and torch.equal(b, out)
    h, v, rel = ref.norm(x, res, None, 1e-6)
    ref.within(out, v, rel, "out")


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_norm_of_extreme_rows(dev, dtype):
    """Zeros, tiny and huge rows, an infinity, a NaN: each stays in its row."""
    x = normal((8, 392), dtype, dev, 5)
    top = torch.finfo(dtype).max
    x[0] = 0
    x[1] = 1e-30 if dtype == BF16 else 6e-8
    x[2] = x[2] * (1e37 if dtype == BF16 else 1e4)
    x[3] = top
    x[4, 100] = float("inf")
    x[5, 300] = float("nan")
    x[6, ::3] = -top
    out, q, scale = torch.empty_like(x), torch.empty_like(x, dtype=ref.E4M3), torch.empty((8, 4), device=dev)
    m.lora_rms_norm(x, None, 1e-5, out=out, q=q, q_scale=scale)
    h, v, rel = ref.norm(x, None, None, 1e-5)
    fine = [0, 1, 2, 3, 6, 7]
    ref.within(out[fine], v[fine], rel, "out")
    ref.check_rows8(q[fine], scale[fine], v[fine], rel, "q")
    assert (q[0].float() == 0).all() and (scale[0] == 2.0 ** -126).all()
    nan = torch.isnan(out[4])
    assert nan[100] and nan.sum() == 1 and (out[4][~nan] == 0).all()
    assert torch.isnan(q[4].float()[:128]).all() and (q[4].float()[128:] == 0).all()  # the block's scale is NaN
    assert torch.isnan(out[5]).all() and torch.isnan(q[5].float()).all() and torch.isnan(scale[5]).all()


@pytest.mark.parametrize("rows, width", [(1, 8), (1, 1024), (3, 120), (2, 136), (33, 11008), (5, 2744), (2, 70008), (1500, 264)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("gate", [False, True])
def test_quantize(dev, rows, width, dtype, gate):
    both = normal((rows, 2 * width + 8), dtype, dev, 7, 3.0)
    both[:, ::29] *= 12
    x, g = both[:, :width], both[:, width + 8:] if gate else None
    out, out_wide = framed(rows, width, dtype, dev, 8)
    q, q_wide = framed(rows, width, ref.E4M3, dev, 8)
    scale, scale_wide = framed(rows, -(-width // 128), torch.float32, dev, 1)
    m.lora_quantize(x, q, scale, gate=g, out=out)
    v, rel = ref.gated(x, g)
    ref.within(out, v, rel, "out")
    ref.check_rows8(q, scale, v, rel, "q")
    assert untouched(out_wide, width) and untouched(q_wide, width) and untouched(scale_wide, scale.shape[1])
    alone = torch.empty_like(out)
    m.lora_quantize(x, gate=g, out=alone)
    assert torch.equal(alone, out)
    q2, s2 = torch.empty_like(q), torch.empty_like(scale)
    m.lora_quantize(x, q2, s2, gate=g)
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, scale)
    for into in ("x", "gate") if gate else ("x",):  # in place
        a, b = x.clone(), g.clone() if gate else None
        m.lora_quantize(a, gate=b, out=a if into == "x" else b)
        assert torch.equal(a if into == "x" else b, out)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantize_of_extreme_blocks(dev, dtype):
    x = normal((1, 7 * 128), dtype, dev, 9)
    b = x.view(7, 128)
    b[0] = 0
    b[1] = 1e-39 if dtype == BF16 else 6e-8  # bf16: below the smallest scale's share
    b[2] = torch.finfo(dtype).max
    b[3, 5] = float("-inf")
    b[4, 9] = float("nan")
    b[5] = 0
    b[5, 127] = 1
    q, scale = torch.empty_like(x, dtype=ref.E4M3), torch.empty((1, 7), device=dev)
    m.lora_quantize(x, q, scale)
    f, s = q.float().view(7, 128), scale[0]
    assert (f[0] == 0).all() and s[0] == 2.0 ** -126
    ref.check_rows8(torch.cat([q[:, :384], q[:, 640:]], 1), torch.cat([scale[:, :3], scale[:, 5:]], 1),
                    torch.cat([x[:, :384], x[:, 640:]], 1).double(), 0.0, "q")
    assert s[3] == float("inf") and torch.isnan(f[3, 5]) and (f[3, :5] == 0).all() and (f[3, 6:] == 0).all()
    assert torch.isnan(f[4]).all() and torch.isnan(s[4])
    assert (f[5, :127] == 0).all() and f[5, 127] == 448


def test_gate_of_all_sizes(dev):
    """Gates over fp32's range of exp, and infinities."""
    g = torch.cat([torch.linspace(-86, 90, 1008), torch.tensor([-100.0, -1e4, 1e4, float("inf"), 0.0, -0.0, 1e-30, -3e-5])])
    g = g.to(BF16).to(dev)[None]
    x, out = torch.full_like(g, 3.0), torch.empty_like(g)
    m.lora_quantize(x, gate=g, out=out)
    v, rel = ref.gated(x, g)
    ref.within(out, v, rel, "out")
    g[0, 0], g[0, 1] = float("-inf"), float("nan")
    m.lora_quantize(x, gate=g, out=out)
    assert torch.isnan(out[0, :2]).all()


def test_empty_and_many_rows(dev):
    before = m.launch_count()
    none = torch.empty((0, 64), dtype=BF16, device=dev)
    m.lora_rms_norm(none, out=torch.empty_like(none))
    m.lora_quantize(none, out=torch.empty_like(none))
    assert m.launch_count() == before
    rows = 70001  # beyond a grid's 65535
    x = torch.arange(rows, device=dev, dtype=torch.float32)[:, None].repeat(1, 8).to(BF16)
    out, q, scale = torch.empty_like(x), torch.empty_like(x, dtype=ref.E4M3), torch.empty((rows, 1), device=dev)
    m.lora_rms_norm(x, out=out)
    ref.within(out, *ref.norm(x, None, None, 1e-5)[1:], "out")
    m.lora_quantize(x, q, scale)
    assert (q[1:].float() == 448).all()


def test_graph_replay_on_another_stream(dev):
    x, res = normal((9, 4096), BF16, dev, 1), normal((9, 4096), BF16, dev, 2)
    out, sums = torch.empty_like(x), torch.empty_like(x)
    q, scale = torch.empty_like(x, dtype=ref.E4M3), torch.empty((9, 32), device=dev)
    norm = m.RmsNorm(x, None, 1e-5, residual=res, residual_out=sums, out=out, q=q, q_scale=scale)
    norm()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        norm()
    x.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    h, v, rel = ref.norm(x, res, None, 1e-5)
    ref.within(out, v, rel, "out")
    ref.check_rows8(q, scale, v, rel, "q")
