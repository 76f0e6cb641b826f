"""lora_sample where its temperatures leave fp32's normal numbers."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
from test_gpu_step_rows import dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("temperature", [2.0 ** -126, 2.0 ** -127, 1e-40, 2.0 ** -149])
@pytest.mark.parametrize("min_p", [0.0, 0.2])
def test_temperatures_below_the_normal_numbers_count_as_the_smallest(dev, temperature, min_p):  # noqa: F811
    x = torch.tensor([0.0, -0.5, -1.0, -2.0, -3.0]).repeat(16, 1) * 2.0 ** -126
    u = (torch.arange(16) + 0.37) / 16
    t, lp = torch.empty(16, dtype=torch.int32, device=dev), torch.empty(16, device=dev)
    m.lora_sample(t, x.to(dev), u.to(dev), temperature=torch.full((16,), temperature, device=dev),
                  min_p=torch.full((16,), min_p, device=dev), logprob=lp)
    want, want_lp, margin = ref.sample(x, u, temperature=torch.full((16,), 2.0 ** -126), min_p=torch.full((16,), min_p))
    assert min(margin) > 2.0 ** -30 and t.tolist() == want
    for got, lq in zip(lp.tolist(), want_lp):
        assert abs(got - lq) <= 8 * ref.U * (1 + abs(lq)) + 4 * ref.U * abs(lq)


@pytest.mark.parametrize("vocab", [5, 3001])
def test_a_difference_beyond_fp32_has_no_weight(dev, vocab):  # noqa: F811
    """However large the temperature: (logit - the largest) is a number of fp32, or -inf."""
    x = torch.full((1, vocab), -3e38)
    x[0, 3] = 3e38
    t = torch.empty(1, dtype=torch.int32, device=dev)
    for temperature in (1e38, 3e38, float("inf")):
        m.lora_sample(t, x.to(dev), torch.tensor([0.9999], device=dev), temperature=torch.tensor([temperature], device=dev))
        assert int(t) == 3
