"""lora_fp8_matmul against its definition in 64 bits (step_ref)."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
from test_gpu_step_rows import BF16, FP16, dev, framed, untouched  # noqa: F401

pytestmark = pytest.mark.gpu


def rows8(rows, width, dev, seed, block_rows=1):  # noqa: F811
    """e4m3 values of all sizes and scales that differ from block to block."""
    g = torch.Generator(device=dev).manual_seed(seed)
    q = torch.empty((rows, width), device=dev).normal_(0, 80, generator=g).clamp_(-448, 448).to(ref.E4M3)
    s = torch.empty((-(-rows // block_rows), -(-width // 128)), device=dev).normal_(0, 1, generator=g).exp_() * 1e-3
    return q, s


def check(dev, rows, d_in, d_out, dtype, seed=0, pad=0):  # noqa: F811
    x, xs = rows8(rows, d_in, dev, seed + 1)
    w, ws = rows8(d_out, d_in, dev, seed + 2, 128)
    if pad:  # wider arrays, NaN behind what belongs to the product
        wide = torch.full((rows, d_in + 16 * pad), float("nan"), device=dev).to(ref.E4M3)
        wide[:, :d_in] = x
        x = wide[:, :d_in]
        wide = torch.full((d_out, d_in + 16 * pad), float("nan"), device=dev).to(ref.E4M3)
        wide[:, :d_in] = w
        w = wide[:, :d_in]
        xs, ws = (torch.cat([t, torch.full((t.shape[0], pad), float("nan"), device=dev)], 1)[:, : t.shape[1]] for t in (xs, ws))
    y, y_wide = framed(rows, d_out, dtype, dev, 8 * pad)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    m.lora_fp8_matmul(y, x, xs, w, ws, st)
    want, off = ref.matmul(x, xs, w, ws)
    assert int(st.item()) == 0
    err = (y.double() - want).abs()
    bound = want.abs() * (torch.finfo(dtype).eps / 2) + off * (1 + torch.finfo(dtype).eps) + ref.STEP[dtype]
    assert bool((err <= bound).all()), f"{int((err > bound).sum())} of {err.numel()} off, worst {float((err / bound).max()):.3g} bounds"
    assert untouched(y_wide, d_out)
    return x, xs, w, ws, y


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("d_in, d_out", [(512, 384), (2064, 1000)])
def test_rows(dev, rows, d_in, d_out):  # noqa: F811
    check(dev, rows, d_in, d_out, BF16)


@pytest.mark.parametrize("d_in", [16, 32, 112, 128, 144, 256, 272, 640, 1040, 4096, 11008])
@pytest.mark.parametrize("rows", [1, 40, 150])
def test_depths(dev, d_in, rows):  # noqa: F811
    check(dev, rows, d_in, 264, FP16)


@pytest.mark.parametrize("d_out", [8, 16, 120, 128, 136, 256, 264, 1032, 5120])
@pytest.mark.parametrize("rows", [1, 24, 130, 700])
def test_widths(dev, d_out, rows):  # noqa: F811
    check(dev, rows, 400, d_out, BF16)


@pytest.mark.parametrize("rows, d_in, d_out", [(1, 4096, 4096), (32, 4096, 11008), (60, 8192, 1024), (256, 8192, 2048), (2500, 1024, 5120),
                                               (4000, 256, 640)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_real_sizes(dev, rows, d_in, d_out, dtype):  # noqa: F811
    check(dev, rows, d_in, d_out, dtype)


@pytest.mark.parametrize("rows", [1, 5, 90, 300])
@pytest.mark.parametrize("pad", [1, 3])
def test_strided(dev, rows, pad):  # noqa: F811
    check(dev, rows, 656, 392, BF16, pad=pad)


@pytest.mark.parametrize("rows", [3, 70, 400])
def test_the_same_bits_again_and_in_a_graph(dev, rows):  # noqa: F811
    x, xs, w, ws, y = check(dev, rows, 2048, 1024, BF16)
    first = y.clone()
    call = m.Fp8Matmul(y, x, xs, w, ws)
    for _ in range(3):
        y.fill_(0)
        call()
        assert torch.equal(y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    xs.mul_(2)  # by a power of two: every rounding the same
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first * 2)


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_nan_and_infinity_stay_in_their_rows_and_columns(dev, rows):  # noqa: F811
    x, xs, w, ws, y = check(dev, rows, 512, 256, BF16)
    clean = y.clone()
    x.view(torch.uint8)[1, 77] = 0x7F
    m.lora_fp8_matmul(y, x, xs, w, ws)
    assert torch.isnan(y[1]).all() and torch.equal(y[2:], clean[2:]) and torch.equal(y[0], clean[0])
    x.view(torch.uint8)[1, 77] = 0
    xs[0, 2] = float("inf")
    m.lora_fp8_matmul(y, x, xs, w, ws)
    assert not torch.isfinite(y[0]).any() and torch.equal(y[2:], clean[2:])
    xs[0, 2] = 1
    w.view(torch.uint8)[200, 300] = 0xFF
    m.lora_fp8_matmul(y, x, xs, w, ws)
    assert torch.isnan(y[:, 200]).all() and torch.equal(y[2:, :200], clean[2:, :200]) and torch.equal(y[2:, 201:], clean[2:, 201:])


def test_no_rows_launch_nothing(dev):  # noqa: F811
    before = m.launch_count()
    w, ws = rows8(64, 128, dev, 1, 128)
    e = torch.empty
    m.lora_fp8_matmul(e((0, 64), dtype=BF16, device=dev), e((0, 128), dtype=ref.E4M3, device=dev), e((0, 1), device=dev), w, ws)
    assert m.launch_count() == before
