"""The time-out path of the 8-bit product's kernels, made to run out without any fault: a limit of a few nanoseconds
(lora_test_set_wait_limit_ns) ends a wait unless its data is already there. The loads and products do end, just after the wait
stopped looking, and the CTA waits for them; the call reports TIMEOUT and leaves every element of y untouched or right; the
next call, with the limit of 2 s again, is right. Longer limits fall into the middle of a call."""
import time

import pytest
import torch

import adapter_gemv_gb300 as m
from test_gpu_step_matmul import check
from test_gpu_step_rows import BF16, FP16, dev  # noqa: F401

pytestmark = pytest.mark.gpu


# few rows with K over a cluster of 8, of 3 and over none; many rows with tiles of one and of several turns an SM
@pytest.mark.parametrize("rows, d_in, d_out", [(4, 4096, 1024), (20, 2064, 6000), (64, 1040, 12800), (300, 1024, 4096), (1000, 512, 8192)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_wait_that_runs_out(dev, rows, d_in, d_out, dtype):  # noqa: F811
    x, xs, w, ws, want = check(dev, rows, d_in, d_out, dtype)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    y = torch.empty_like(want)
    call = m.Fp8Matmul(y, x, xs, w, ws, st)
    torch.cuda.synchronize()
    late = 0
    for limit in (2, 2, 300, 900, 1500, 3000, 10000):
        y.fill_(-77.0), st.zero_()
        m.lora_test_set_wait_limit_ns(limit)
        try:
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            took = time.perf_counter() - t0
        finally:
            m.lora_test_set_wait_limit_ns(0)
        got = int(st.item())
        assert got in (0, m.STATUS_TIMEOUT)
        right = y == want
        assert bool((right | (y == -77.0)).all()), f"limit {limit}: {int((~right & (y != -77.0)).sum())} elements neither untouched nor right"
        assert got or bool(right.all()), f"limit {limit}: rows left out and nothing reported"
        assert took < 5
        late += limit == 2 and got == m.STATUS_TIMEOUT
        # the default limit again
        y.fill_(-77.0), st.zero_()
        call()
        assert torch.equal(y, want) and int(st.item()) == 0
    assert late == 2, "no wait gave up with a limit of 2 ns"


def test_a_call_that_runs_out_beside_one_that_does_not(dev):  # noqa: F811
    """Two streams, the limit of one of them short: the other's result is right."""
    x, xs, w, ws, want = check(dev, 48, 4096, 2048, BF16)
    x2, xs2, w2, ws2, want2 = check(dev, 400, 1024, 4096, BF16, seed=9)
    st, st2 = (torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(2))
    a, b = m.Fp8Matmul(want.clone().zero_(), x, xs, w, ws, st), m.Fp8Matmul(want2.clone().zero_(), x2, xs2, w2, ws2, st2)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.keep[0].fill_(5), b.keep[0].fill_(5), st.zero_(), st2.zero_()
        torch.cuda.synchronize()
        m.lora_test_set_wait_limit_ns(2)
        try:
            a(one)
        finally:
            m.lora_test_set_wait_limit_ns(0)
        b(two)
        torch.cuda.synchronize()
        assert torch.equal(b.keep[0], want2) and int(st2.item()) == 0
        assert int(st.item()) == m.STATUS_TIMEOUT and bool(((a.keep[0] == want) | (a.keep[0] == 5)).all())
