"""The chain between the projections, each call's output against its definition in 64 bits from what the call before it wrote: norm,
8-bit product, adapters, gate, 8-bit product."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
import workloads as W
from test_gpu_step_rows import BF16, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def check_product(y, want, off, what):
    bound = want.abs() * (torch.finfo(y.dtype).eps / 2) + off * (1 + torch.finfo(y.dtype).eps) + ref.STEP[y.dtype]
    wrong = (y.double() - want).abs() > bound
    assert not bool(wrong.any()), f"{what}: {int(wrong.sum())} of {wrong.numel()} off"


@pytest.mark.parametrize("rows", [1, 3, 40, 300])
def test_every_call_of_the_chain(dev, rows):  # noqa: F811
    d, mlp, rank = 640, 1152, 8
    g = W.generator(23, dev)
    weights = [(torch.randn(o, i, generator=g, device=dev) * 60).clamp(-448, 448).to(ref.E4M3) for i, o in ((d, 2 * mlp), (mlp, d))]
    scales = [torch.rand(-(-w.shape[0] // 128), -(-w.shape[1] // 128), generator=g, device=dev) * 1e-3 for w in weights]
    pool = W.stacked_pool(num_slots=3, num_layers=1, r_max=rank, d_in=d, d_out=2 * mlp, dtype=BF16, gen=g, device=dev)
    handle, slot = m.make_pool(pool), torch.arange(rows, dtype=torch.int32, device=dev) % 4 - 1
    e = lambda n, t=BF16: torch.empty((rows, n), dtype=t, device=dev)  # noqa: E731
    rows8 = lambda n: (e(n, ref.E4M3), e(-(-n // 128), torch.float32))  # noqa: E731
    x, res = (torch.randn((rows, d), generator=g, device=dev).to(BF16) for _ in range(2))
    weight = 1 + 0.2 * torch.randn(d, generator=g, device=dev).to(BF16)
    sums, h, h8, y, act, a8, z = e(d), e(d), rows8(d), e(2 * mlp), e(mlp), rows8(mlp), e(d)
    st = torch.zeros(1, dtype=torch.int32, device=dev)

    m.lora_rms_norm(x, weight, 1e-5, residual=res, residual_out=sums, out=h, q=h8[0], q_scale=h8[1])
    total, v, rel = ref.norm(x, res, weight, 1e-5)
    ref.within(sums, total, ref.U, "sums")
    ref.within(h, v, rel, "h")
    ref.check_rows8(*h8, v, rel, "h in 8 bits")

    m.lora_fp8_matmul(y, *h8, weights[0], scales[0], st)
    check_product(y, *ref.matmul(*h8, weights[0], scales[0]), "y, the base product")
    base = y.clone()
    m.lora_bgmv(y, h, handle, slot, 0, e(rank, torch.float32), st)
    # y + s (h A) B, rows of slot -1 as they were. In fp32: sums of d and of rank products, the scale, the addition to y
    a, b, s = pool.a_t[:, 0].double(), pool.b[:, 0].double(), pool.scale.double()
    want, off = base.double(), torch.zeros((rows, 2 * mlp), dtype=torch.float64, device=dev)
    for k in range(3):
        at = slot == k
        want[at] += s[k] * (h[at].double() @ a[k].t()) @ b[k]
        off[at] = s[k] * (h[at].double().abs() @ a[k].abs().t()) @ b[k].abs() * ((d + rank + 2) * ref.U) + want[at].abs() * ref.U
    check_product(y, want, off, "y, with the adapters")
    assert torch.equal(y[slot < 0], base[slot < 0])

    up, gate = y[:, mlp:], y[:, :mlp]
    m.lora_quantize(up, *a8, gate=gate, out=act)
    v, rel = ref.gated(up, gate)
    ref.within(act, v, rel, "act")
    ref.check_rows8(*a8, v, rel, "act in 8 bits")

    m.lora_fp8_matmul(z, *a8, weights[1], scales[1], st)
    check_product(z, *ref.matmul(*a8, weights[1], scales[1]), "z")
    assert int(st.item()) == 0
