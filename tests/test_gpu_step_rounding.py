"""How the quantiser rounds: q is the fp32 quotient v / scale, correctly rounded, to the nearest e4m3, ties to even.
Every value here that is compared bit for bit is worked out on the CPU, or by division without a shortcut."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
from test_gpu_step_rows import BF16, FP16, dev, normal  # noqa: F401

pytestmark = pytest.mark.gpu


def quantized(x, gate=None):
    q, s = torch.empty_like(x, dtype=ref.E4M3), torch.empty((x.shape[0], -(-x.shape[1] // 128)), device=x.device)
    m.lora_quantize(x, q, s, gate=gate)
    return q, s


def quotients(x, scale):
    """fp32 x / scale as e4m3, on the CPU (its division is correctly rounded; 448 is the largest)."""
    spread = scale.cpu().repeat_interleave(128, 1)[:, : x.shape[1]]
    return (x.cpu().float() / spread).clamp(-448, 448).to(ref.E4M3)


def e4m3_64(z):
    """64-bit z to the nearest e4m3, ties to even, from the format's steps."""
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(z / step) * step, -448, 448)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ties_go_to_the_even_neighbour(dev, dtype):  # noqa: F811
    """A block with maximum 49 has scale 7/64, and 7/64 (2 k + 1) / 2 2^e is half way between two e4m3 values, exactly."""
    half = torch.tensor([(2 * k + 1) / 2 * 2.0 ** e for e in range(-6, 4) for k in range(8, 16)])
    x = torch.zeros((2, 256))
    x[:, 0], x[0, 1:81], x[1, 1:81] = 49.0, half * 7 / 64, -half * 7 / 64
    x[:, 128] = 49.0 * 2.0 ** -5  # the same with a smaller scale
    x[:, 129:209] = x[:, 1:81] * 2.0 ** -5
    x = x.to(dtype).to(dev)
    q, scale = quantized(x)
    assert (scale[:, 0] == 7 / 64).all() and (scale[:, 1] == 7 / 2048).all()
    z = x.double().cpu() / scale.double().cpu().repeat_interleave(128, 1)
    exact = z[0, 1:81] == half.double()  # (fp16 holds the smallest in fewer bits)
    assert int(exact.sum()) >= 70
    assert torch.equal(q.cpu().float().double(), e4m3_64(z))
    even = e4m3_64(half.double())[exact].to(ref.E4M3)
    assert (even.view(torch.uint8) & 1 == 0).all()
    assert torch.equal(q.cpu()[0, 1:81].view(torch.uint8)[exact], even.view(torch.uint8))


@pytest.mark.parametrize("rows, width", [(1, 8), (7, 4096), (600, 5120), (5, 1000)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_the_quotient_is_a_division(dev, rows, width, dtype):  # noqa: F811
    x = normal((rows, width), dtype, dev, rows + width)
    q, scale = quantized(x)
    blocks = torch.nn.functional.pad(x.cpu().float(), (0, -width % 128)).reshape(rows, -1, 128).abs().amax(-1)
    assert torch.equal(scale.cpu(), blocks / torch.full_like(blocks, 448))
    assert torch.equal(q.cpu().float(), quotients(x, scale).float())


@pytest.mark.parametrize("dtype, bits", [(BF16, 8), (FP16, 11)])
def test_every_pair_of_16_bit_significands(dev, dtype, bits):  # noqa: F811
    """A block's largest value m and a value v: all significands of both, v down to 2^-10 of m."""
    n = 2 ** (bits - 1)
    sig = torch.arange(n, 2 * n, dtype=torch.float32)
    values = (sig[None] * torch.exp2(-torch.arange(0.0, 11.0))[:, None]).reshape(-1)  # 11 n of them, 126 a block
    values = torch.nn.functional.pad(values, (0, -len(values) % 126)).reshape(-1, 126)
    for m0 in range(0, n, 128):
        top = sig[m0:m0 + 128]
        x = torch.zeros((top.numel(), values.shape[0], 128))
        x[:, :, 0] = 2 * top[:, None]  # above every value
        x[:, :, 2:] = values
        x = (x / (2 * n)).to(dtype).reshape(top.numel(), -1)
        q, scale = quantized(x.to(dev))
        assert torch.equal(q.cpu().float(), quotients(x, scale).float())


def test_scales_of_all_sizes(dev):  # noqa: F811
    """Blocks from fp32's smallest numbers to its largest, each with values down to nothing."""
    g = torch.Generator().manual_seed(3)
    sizes = torch.cat([torch.exp2(torch.arange(-133.0, 128.0)), torch.tensor([3.3e38, 1.2e-38, 5.3e-36, 5.2e-36])])
    x = torch.empty((sizes.numel(), 128)).uniform_(-1, 1, generator=g) * torch.exp2(-16 * torch.rand((sizes.numel(), 128), generator=g))
    x[:, 0] = 1
    x = (x.double() * sizes.double()[:, None]).to(BF16).to(dev)
    q, scale = quantized(x)
    amax = x.cpu().float().abs().amax(1, keepdim=True)
    assert torch.equal(scale.cpu(), torch.maximum(amax / torch.full_like(amax, 448), torch.tensor(2.0 ** -126)))
    assert torch.equal(q.cpu().float(), quotients(x, scale).float())


# silu(gate) x in fp32: expf is documented to 1 ulp, at most 2 u of its value. A negative gate: its product with that 3 u, 1 + exp 2 u at
# most, the quotient 1 u, the product with x 1 u: 7 u, and a little for their products. A positive one: 4 u.
GATED = 7.001 * ref.U


@pytest.mark.parametrize("dtype, std", [(FP16, 4.0), (BF16, 1.5), (BF16, 12.0)])
def test_gated_values_are_off_by_a_few_roundings(dev, dtype, std):  # noqa: F811
    """Whatever the gate's size, in 16 bits and in 8: no value is rounded the wrong way that is further than that from
    the border between its neighbours."""
    rows, width = 2048, 8192
    x, g = normal((rows, width), dtype, dev, 31, 1.5), normal((rows, width), dtype, dev, 32, std)
    out, q = torch.empty_like(x), torch.empty_like(x, dtype=ref.E4M3)
    scale = torch.empty((rows, width // 128), device=dev)
    m.lora_quantize(x, q, scale, gate=g, out=out)
    v = x.double() * g.double() / (1 + torch.exp(-g.double()))
    bits = {BF16: 8, FP16: 11}[dtype]
    half = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=torch.finfo(dtype).tiny))) - bits)
    bound = half + v.abs() * GATED
    off = (out.double() - v).abs()
    assert bool((off <= bound).all()), f"{int((off > bound).sum())} of out off, worst {float((off / bound).max()):.6f}"
    blocks = v.reshape(rows, -1, 128)
    amax = torch.maximum(blocks.abs().amax(-1) / 448, torch.full_like(scale, 2.0 ** -126, dtype=torch.float64))
    assert bool(((scale.double() - amax).abs() <= amax * (GATED + ref.U)).all())
    z = (blocks / scale.double()[..., None]).reshape(rows, width)
    off = (q.double() - z).abs()
    half = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 4)
    # (the values' error, the quotient's rounding; behind the largest of a binade the next one's step begins)
    bound = half + z.abs() * (GATED + 1.001 * ref.U)
    assert bool((off <= bound).all()), f"{int((off > bound).sum())} of q off, worst {float((off / bound).max()):.6f}"
