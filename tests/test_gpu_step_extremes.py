"""The norm at the ends of fp32's range, against its definition in 64 bits (step_ref)."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
from test_gpu_step_rows import BF16, dev, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [520, 8200, 16400])
@pytest.mark.parametrize("in_place", [False, True])
def test_sums_of_two_finite_rows_beyond_fp32(dev, width, in_place):  # noqa: F811
    """x + residual passes fp32's largest number in some places: its norm is finite, the sum itself rounds to an infinity."""
    top = torch.finfo(BF16).max
    x, res = normal((5, width), BF16, dev, 1, 1e37), normal((5, width), BF16, dev, 2, 1e37)
    x[0, 3], res[0, 3] = top, top
    x[1, ::2], res[1, ::2] = -top, -top
    x[2], res[2] = top, top
    x[3, width - 1], res[3, width - 1] = top, 0.9 * top
    x[3, 5], res[3, 5] = top, -top  # 0
    w = normal((width,), BF16, dev, 3, 0.3) + 1
    h, v, rel = ref.norm(x, res, w, 1e-5)
    out, sums = torch.empty_like(x), res.clone() if in_place else torch.empty_like(x)
    q, scale = torch.empty_like(x, dtype=ref.E4M3), torch.empty((5, -(-width // 128)), device=dev)
    m.lora_rms_norm(x, w, 1e-5, residual=sums if in_place else res, residual_out=sums, out=out, q=q, q_scale=scale)
    assert torch.isfinite(out.float()).all() and torch.isfinite(scale).all() and torch.isfinite(q.float()).all()
    ref.within(out, v, rel, "out")
    ref.check_rows8(q, scale, v, rel, "q")
    ref.within(sums, h, ref.U, "residual")
    assert torch.isinf(sums[2]).all() and sums[0, 3] == float("inf") and sums[1, 0] == -float("inf") and sums[3, 5] == 0


@pytest.mark.parametrize("eps", [1e25, 1e30, 1e38, 3.3e38])
def test_an_eps_that_counts_beside_the_largest_squares(dev, eps):  # noqa: F811
    x = normal((4, 264), BF16, dev, 4)
    for i, size in enumerate((6e18, 1e19, 3e12, 1.0)):
        x[i] = (x[i].float() * size).to(BF16)
    out = torch.empty_like(x)
    m.lora_rms_norm(x, None, eps, out=out)
    ref.within(out, *ref.norm(x, None, None, eps)[1:], "out")


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30])
def test_the_smallest_eps(dev, eps):  # noqa: F811
    """Rows whose squares are as small as eps, or leave fp32's range downwards: each square and their sums are off by
    4 x 2^-150 at most, 2^-22 of the sum with eps, half of that behind the root."""
    x = normal((5, 392), BF16, dev, 6)
    for i, size in enumerate((2.0 ** -63, 2.0 ** -66, 2.0 ** -80, 2.0 ** -50, 0.0)):
        x[i] = (x[i].float() * size).to(BF16)
    out = torch.empty_like(x)
    m.lora_rms_norm(x, None, eps, out=out)
    _, v, rel = ref.norm(x, None, None, eps)
    ref.within(out, v, rel + 2.0 ** -23, "out")
