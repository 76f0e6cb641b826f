"""Calls of the norm, the 8-bit rows, the product and the sampling that the header does not allow, beside those of
test_step_abi: refused on the host before anything is launched (CPU only)."""
import pytest

import adapter_gemv_gb300 as m
from test_serve_abi import L  # noqa: F401
from test_step_abi import call

# Every array at an address of its own.
A = [0x10000000 + (i << 24) for i in range(16)]
NORM = dict(num_rows=3, width=264, dtype=0, eps=1e-5, x=A[0], residual=A[1], weight=A[2], residual_out=A[3], out=A[4], q=A[5], q_scale=A[6],
            ldx=264, ldr=264, ldro=264, ldo=264, ldq=264, lds=3)
QUANT = dict(num_rows=3, width=264, dtype=1, x=A[0], gate=A[1], out=A[2], q=A[3], q_scale=A[4], ldx=264, ldg=264, ldo=264, ldq=264, lds=3)
MATMUL = dict(num_rows=3, d_in=272, d_out=136, dtype=0, x=A[0], x_scale=A[1], w=A[2], w_scale=A[3], y=A[4], ldx=272, ldxs=3, ldw=272, ldws=3,
              ldy=136)
SAMPLING = dict(num_rows=3, vocab=1001, dtype=2, num_requests=3, logits=A[0], ld=1001, row_request=A[1], uniform=A[2], temperature=A[3],
                top_k=A[4], top_p=A[5], min_p=A[6], token=A[7], logprob=A[8])


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 2.0 ** -127, 2.0 ** -126 * (1 - 2.0 ** -23)])
def test_an_eps_below_fp32s_normal_numbers(L, eps):  # noqa: F811
    """Squares as small as such an eps have no 24 bits."""
    assert call(L, "norm", dict(eps=eps), NORM) == m.ERR_SHAPE
    assert call(L, "norm", dict(eps=2.0 ** -126, num_rows=0), NORM) == 0


@pytest.mark.parametrize("name, base, out, others", [
    ("norm", NORM, "q", ["x", "residual", "weight", "out", "residual_out"]),
    ("norm", NORM, "q_scale", ["x", "residual", "weight", "out", "residual_out", "q"]),
    ("norm", NORM, "out", ["weight", "residual_out"]), ("norm", NORM, "residual_out", ["weight"]),
    ("quant", QUANT, "q", ["x", "gate", "out"]), ("quant", QUANT, "q_scale", ["x", "gate", "out", "q"]),
    ("matmul", MATMUL, "y", ["x", "w", "x_scale", "w_scale"]),
    ("sampling", SAMPLING, "token", ["logits", "row_request", "uniform", "temperature", "top_k", "top_p", "min_p"]),
    ("sampling", SAMPLING, "logprob", ["logits", "row_request", "uniform", "temperature", "top_k", "top_p", "min_p", "token"])])
def test_an_output_over_another_array(L, name, base, out, others):  # noqa: F811
    """Other rows' CTAs would read what has been written."""
    for other in others:
        assert call(L, name, {out: base[other]}, base) == m.ERR_SHAPE, (out, other)


@pytest.mark.parametrize("num_rows, d_out", [(2 ** 31 - 1, 264), (2 ** 28 + 1, 2048), (2 ** 20, 2 ** 20)])
def test_a_product_of_more_tiles_than_a_grid_counts(L, num_rows, d_out):  # noqa: F811
    """(y would be a terabyte or more)"""
    assert call(L, "matmul", dict(num_rows=num_rows, d_out=d_out, ldy=d_out), MATMUL) == m.ERR_SHAPE
