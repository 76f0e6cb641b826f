"""lora_kv_attention over values that are infinities or NaN: the outputs are what the definition in 64 bits makes them."""
import pytest
import torch

import serve_ref as ref
from test_gpu_serve_attention import Case, dev, with_rows  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def put(c, request, token, value, elements):
    pt = c.k.shape[2]
    c.v[c.layer, int(c.table[request, token // pt]), token % pt, :, elements] = value


def check_kinds(c):
    """Every finite output within its tolerance; infinities where the definition has them, with their sign; NaN likewise."""
    c.run()
    assert int(c.status.item()) == 0
    d = c.q.shape[1] // c.hq
    want, lse, tol, ltol = ref.attention(c.q.reshape(-1, c.hq, d), c.k, c.v, c.layer, c.table, c.request, c.position, c.scale,
                                         c.window)
    out = c.out.reshape(-1, c.hq, d).double()
    ref.assert_within(c.lse, lse, ltol, "lse")
    fine = torch.isfinite(want)
    assert not fine.all() and fine.any()
    ref.assert_within(out[fine], want[fine], tol[fine], "out")
    got, want = out[~fine], want[~fine]
    assert torch.equal(got.isnan(), want.isnan()), f"{int((got.isnan() != want.isnan()).sum())} of {want.numel()} NaN differ"
    assert torch.equal(got[~got.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_one_token_with_an_infinite_value(dev, dtype, value):  # noqa: F811
    c = Case(dev, [1, 1, 2, 3], 4, 2, 64, dtype=dtype)
    for r in range(4):
        put(c, r, 0, value, [0, 9, 63])
    check_kinds(c)


@pytest.mark.parametrize("hq, hk, d, pt, dtype", [
    (4, 4, 128, 16, torch.bfloat16), (8, 1, 128, 32, torch.float16), (16, 2, 64, 16, torch.bfloat16),
    (15, 5, 80, 24, torch.float16), (24, 2, 256, 8, torch.bfloat16), (40, 2, 96, 16, torch.float16), (3, 1, 8, 1, torch.bfloat16)])
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("q_std", [1.0, 30.0])
def test_infinite_values(dev, hq, hk, d, pt, dtype, window, q_std):  # noqa: F811
    """In first, middle and last tokens, in rows that are split over the GPU, whatever the weight (with q_std = 30 most
    are below fp32's smallest number, but none is 0)."""
    lens = [1, 2, 17, 61, 300, 2500, 9000]
    c = Case(dev, lens, hq, hk, d, pt, dtype=dtype, window=window, q_std=q_std)
    for r, n in enumerate(lens):
        put(c, r, 0, INF, [0])
        put(c, r, n - 1, -INF, [1])
        put(c, r, n // 2, INF, [2, d - 1])
        put(c, r, n // 3, -INF, [2])
        put(c, r, max(0, n - 40), NAN, [3])
    check_kinds(c)


@pytest.mark.parametrize("hq, hk, d, pt, dtype", [
    (4, 2, 128, 16, torch.bfloat16), (15, 5, 80, 24, torch.float16), (32, 16, 64, 16, torch.float16),
    (32, 16, 128, 8, torch.bfloat16), (16, 16, 256, 16, torch.bfloat16), (128, 16, 128, 16, torch.float16),
    (10, 2, 256, 16, torch.bfloat16)])
@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("least", [0, 2600])
def test_infinite_values_in_shared_tiles(dev, hq, hk, d, pt, dtype, window, least):  # noqa: F811
    """Rows that share a tile see the infinities of their own tokens, in a piece's first tile as in later ones."""
    c = Case(dev, [260, 90, 30], hq, hk, d, pt, dtype=dtype, window=window, layers=1)
    rows = [(0, p) for p in range(60, 260)] + [(1, p) for p in range(0, 90)] + [(2, p) for p in range(30)]
    while len(rows) * hk < least:
        rows += [(2, p) for p in range(30)]
    with_rows(c, rows, torch.Generator(device=dev).manual_seed(11))
    for t in (0, 3, 61, 100, 258):
        put(c, 0, t, INF, [t % 7])
    put(c, 0, 70, -INF, [2, 3])
    put(c, 0, 163, NAN, [5])
    put(c, 1, 1, -INF, [0, d - 1])
    put(c, 1, 5, INF, [0])
    put(c, 2, 0, INF, [6])
    put(c, 2, 29, NAN, list(range(d // 2)))
    check_kinds(c)
