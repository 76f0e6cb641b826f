"""Rows beyond what one launch of the quantiser and of the sampling counts: those of the second launch, too."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
from test_gpu_step_rows import BF16, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", [False, True])
def test_quantiser_rows_of_two_launches(dev, gate):  # noqa: F811
    """A block a row, 16 threads a block, threads counted in 31 bits: 134217711 rows of a launch."""
    rows, width = (2 ** 31 - 1 - 256) // 16 + 70, 8
    before = m.launch_count()
    x = torch.arange(rows, device=dev, dtype=torch.int32).bitwise_and_(255).to(BF16)[:, None].repeat(1, width)
    x[:, 1] = -3
    g = torch.full_like(x, 32) if gate else None  # its sigmoid is 1 in fp32
    q, scale, out = torch.empty_like(x, dtype=ref.E4M3), torch.empty((rows, 1), device=dev), torch.empty_like(x)
    m.lora_quantize(x, q, scale, gate=g, out=out)
    assert m.launch_count() == before + 2
    v = x * 32 if gate else x
    assert torch.equal(out, v)
    want = v.abs().amax(1, keepdim=True).float() / torch.full_like(scale, 448)
    assert torch.equal(scale, want)
    for part in (slice(0, 1 << 20), slice(rows - (1 << 20), rows)):  # the launches' first and last rows, and where they meet
        z = v[part].float() / want[part]
        assert torch.equal(q[part].float(), z.clamp(-448, 448).to(ref.E4M3).float())


def test_sampling_rows_of_two_launches(dev):  # noqa: F811
    """2^28 - 1 rows of a launch; most of them are no request's."""
    rows, vocab = 2 ** 28 + 50, 2
    x = torch.zeros((rows, vocab), dtype=BF16, device=dev)
    request = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    some = [0, 1, 2 ** 20, 2 ** 28 - 2, 2 ** 28 - 1, 2 ** 28, rows - 2, rows - 1]
    for i, row in enumerate(some):
        request[row] = i
        x[row, i % 2] = 40
    token, uniform = torch.full((rows,), -7, dtype=torch.int32, device=dev), torch.full((rows,), 0.5, device=dev)
    before = m.launch_count()
    m.lora_sample(token, x, uniform, row_request=request, temperature=torch.ones(len(some), device=dev))
    assert m.launch_count() == before + 2
    assert token[some].tolist() == [i % 2 for i in range(len(some))]
    assert int((token == -7).sum()) == rows - len(some)
