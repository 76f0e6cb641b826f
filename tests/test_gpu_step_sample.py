"""lora_sample against its definition in 64 bits (step_ref): the same tokens, for random numbers that are not at a border
of the definition's own sums (2^-30 of them; the kernel's are off by 2^-36)."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
from test_gpu_step_rows import dev  # noqa: F401

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def check(logits, uniform, dev, **kw):  # noqa: F811
    """kw: the requests' arrays, on the CPU, a row each."""
    rows = logits.shape[0]
    token = torch.full((rows,), 12345, dtype=torch.int32, device=dev)
    logprob = torch.full((rows,), 5.0, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    m.lora_sample(token, logits, uniform.to(dev), logprob=logprob, status=st, **{k: v.to(dev) for k, v in kw.items()})
    want, lp, margin = ref.sample(logits.cpu(), uniform, **kw)
    assert int(st.item()) == 0
    for i in range(rows):
        assert margin[i] > 2.0 ** -30, f"row {i}: the test's own number is at a border"
        assert int(token[i]) == want[i], f"row {i}: {int(token[i])}, {want[i]} wanted"
        if lp[i] == -float("inf"):
            assert float(logprob[i]) == lp[i]
        else:  # y ln 2 in fp32: the sum y + yl, its product, log1p (4 u) and the difference
            assert abs(float(logprob[i]) - lp[i]) <= 8 * ref.U * (1 + abs(lp[i])) + 4 * ref.U * abs(lp[i]), f"row {i}: {float(logprob[i])}, {lp[i]}"
    # without the second output: the same tokens
    again = torch.empty_like(token)
    m.lora_sample(again, logits, uniform.to(dev), **{k: v.to(dev) for k, v in kw.items()})
    assert torch.equal(again, token)
    return token


def make(rows, vocab, dtype, dev, seed, std=3.0):  # noqa: F811
    g = torch.Generator().manual_seed(seed)
    x = torch.empty((rows, vocab)).normal_(0, std, generator=g).to(dtype).to(dev)
    return x, torch.rand(rows, generator=g), g


def limits(rows, vocab, g):
    u = lambda lo, hi: torch.empty(rows).uniform_(lo, hi, generator=g)  # noqa: E731
    some = lambda a, b: torch.where(torch.rand(rows, generator=g) < 0.5, a, b)  # noqa: E731
    return dict(temperature=u(0.2, 2.0), top_k=some(torch.randint(1, vocab + 1, (rows,), generator=g), torch.zeros(rows, dtype=torch.int64)).to(torch.int32),
                top_p=some(u(0.05, 0.99), torch.ones(rows)), min_p=some(u(0.0, 0.3), torch.zeros(rows)))


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 64, 100, 1000, 4097, 32000, 50257, 128001])
@pytest.mark.parametrize("dtype", DTYPES)
def test_all_limits(dev, vocab, dtype):  # noqa: F811
    x, u, g = make(12, vocab, dtype, dev, vocab)
    check(x, u, dev, **limits(12, vocab, g))


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", None])
@pytest.mark.parametrize("vocab", [777, 60001])
def test_each_limit_alone(dev, name, vocab):  # noqa: F811
    x, u, g = make(9, vocab, torch.float32, dev, 5)
    kw = limits(9, vocab, g)
    check(x, u, dev, **({name: kw[name]} if name else {}))


@pytest.mark.parametrize("std", [0.0, 1e-6, 1e-3, 0.3, 30.0, 3e4])
@pytest.mark.parametrize("vocab", [500, 40000])
def test_flat_and_peaked_rows(dev, std, vocab):  # noqa: F811
    x, u, g = make(8, vocab, torch.float32, dev, 11, std)
    check(x, u, dev)
    check(x, u, dev, **limits(8, vocab, g))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [300, 33333])
def test_ties_go_to_the_lowest_id(dev, dtype, vocab):  # noqa: F811
    """A few different values only, zeros of both signs among them: limits and numbers fall inside runs of equal tokens."""
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-2, 3, (20, vocab), generator=g).to(dtype)
    x[:, ::5] = -x[:, ::5]
    kw = dict(top_k=torch.randint(1, vocab, (20,), generator=g).to(torch.int32), top_p=torch.rand(20, generator=g))
    token = check(x.to(dev), torch.rand(20, generator=g), dev, **kw)
    zero = check(x.to(dev), torch.zeros(20), dev, **kw)
    best = torch.sort(x.float(), descending=True, stable=True).indices[:, 0]
    assert (zero.cpu() == best).all() and (token.cpu() >= 0).all()


def test_greedy(dev):  # noqa: F811
    x, u, g = make(6, 5001, torch.bfloat16, dev, 2)
    best = torch.sort(x, descending=True, stable=True).indices[:, 0].to(torch.int32)
    t = torch.tensor([0.0, -1.0, float("nan"), 1.0, 1e-30, 1.0])
    k = torch.tensor([0, 5, 0, 1, 1, 1], dtype=torch.int32)
    token, lp = torch.empty(6, dtype=torch.int32, device=dev), torch.empty(6, device=dev)
    m.lora_sample(token, x, u.to(dev), temperature=t.to(dev), top_k=k.to(dev), logprob=lp)
    assert torch.equal(token, best) and (lp == 0).all()


def test_numbers_at_the_ends_and_outside(dev):  # noqa: F811
    x = torch.tensor([[1.0, 3.0, 2.0, -1.0]]).repeat(8, 1).to(dev)
    u = torch.tensor([0.0, -0.0, 1 - 2.0 ** -24, 1.0, 5.0, -3.0, float("nan"), 1e-40], device=dev)
    token = torch.empty(8, dtype=torch.int32, device=dev)
    m.lora_sample(token, x, u)
    assert token.tolist() == [1, 1, 3, 3, 3, 1, 1, 1]


def test_limits_at_their_ends(dev):  # noqa: F811
    x, _, _ = make(10, 3000, torch.float32, dev, 8)
    u = torch.full((10,), 0.97)
    inf = float("inf")
    check(x, u, dev, top_p=torch.tensor([0.0, -1.0, 1.0, 2.0, float("nan"), 1e-30, 1 - 2.0 ** -24, 0.5, inf, 2.0 ** -140]))
    check(x, u, dev, top_k=torch.tensor([0, -5, 1, 2999, 3000, 3001, 2 ** 31 - 1, -2 ** 31, 2, 10], dtype=torch.int32))
    check(x, u, dev, min_p=torch.tensor([0.0, -1.0, 1.5, inf, float("nan"), 1e-30, 1e-42, 0.9999, 0.01, 1e-5]))
    check(x, u, dev, temperature=torch.tensor([1e30, 3e38, 1e-3, 1e-38, 1e-42, 100.0, 1e-10, 5.0, 1e5, 0.01]))
    flat = torch.zeros((1, 7), device=dev)
    assert int(check(flat, torch.tensor([0.99]), dev, top_p=torch.tensor([0.3]))[0]) == 2  # 3 of 7 tokens reach 0.3 of the mass
    token = torch.empty(1, dtype=torch.int32, device=dev)
    m.lora_sample(token, flat, torch.tensor([0.99], device=dev), temperature=torch.tensor([inf], device=dev))
    assert int(token) == 6
    m.lora_sample(token, flat, torch.tensor([0.99], device=dev), min_p=torch.tensor([1.0], device=dev))
    assert int(token) == 6  # weights equal to the largest reach 1


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan(dev, dtype):  # noqa: F811
    x, u, g = make(8, 2050, dtype, dev, 4)
    inf = float("inf")
    x[0] = -inf
    x[1] = float("nan")
    x[2] = -inf
    x[2, 2049] = -5
    x[3, ::2] = -inf
    x[4, 5], x[4, 1000], x[4, 2000] = inf, inf, inf
    x[5, ::3] = float("nan")
    x[6] = torch.finfo(dtype).min
    x[7, 0], x[7, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
    token = check(x, u, dev)
    assert token[:3].tolist() == [-1, -1, 2049] and int(token[4]) in (5, 1000, 2000)
    check(x, u, dev, **limits(8, 2050, g))


def test_requests_strides_and_skipped_rows(dev):  # noqa: F811
    """Rows of a wider matrix at odd addresses, in another order than the requests'; -1 and numbers that are no request's."""
    g = torch.Generator().manual_seed(6)
    for dtype in DTYPES:
        wide = torch.empty((9, 1013)).normal_(0, 3, generator=g).to(dtype).to(dev)
        x = wide[:, 3:1004]
        n = 4
        kw = {k: v[:n] for k, v in limits(9, 1001, g).items()}
        request = torch.tensor([2, -1, 0, 3, 4, 1, 1, -2, 2], dtype=torch.int32)
        u = torch.rand(9, generator=g)
        token, lp = torch.full((9,), -77, dtype=torch.int32, device=dev), torch.full((9,), 5.0, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        m.lora_sample(token, x, u.to(dev), row_request=request.to(dev), logprob=lp, status=st, **{k: v.to(dev) for k, v in kw.items()})
        real = [0, 2, 3, 5, 6, 8]
        want, _, margin = ref.sample(x[real].cpu(), u[real], **{k: v[request[real].long()] for k, v in kw.items()})
        assert min(margin) > 2.0 ** -30 and token[real].tolist() == want
        assert (token[[1, 4, 7]] == -77).all() and (lp[[1, 4, 7]] == 5).all() and int(st) == m.STATUS_BAD_REQUEST


def test_the_order_of_tokens_says_nothing(dev):  # noqa: F811
    """The sums are of whole numbers: a permuted row gives the permuted token."""
    g = torch.Generator().manual_seed(21)
    x = (torch.randperm(65537, generator=g) * 1e-3).to(dev)[None]  # no two alike
    u = torch.rand(1, generator=g)
    kw = dict(temperature=torch.tensor([3.0], device=dev), top_p=torch.tensor([0.9], device=dev))
    perm = torch.randperm(65537, generator=g).to(dev)
    token, other, lp, lq = (torch.empty(1, dtype=t, device=dev) for t in (torch.int32, torch.int32, torch.float32, torch.float32))
    m.lora_sample(token, x, u.to(dev), logprob=lp, **kw)
    m.lora_sample(other, x[:, perm], u.to(dev), logprob=lq, **kw)
    assert int(perm[int(other)]) == int(token) and float(lp) == float(lq)


def test_the_largest_vocabulary(dev):  # noqa: F811
    x, u, g = make(2, m.SAMPLE_MAX_VOCAB, torch.bfloat16, dev, 31, 0.01)
    check(x, u, dev)
    check(x, u, dev, top_p=torch.tensor([0.5, 0.999]))


def test_graph_replay(dev):  # noqa: F811
    x, u, g = make(5, 9000, torch.float32, dev, 41)
    token, un = torch.empty(5, dtype=torch.int32, device=dev), u.to(dev)
    kw = limits(5, 9000, g)
    call = m.Sample(token, x, un, **{k: v.to(dev) for k, v in kw.items()})
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        u = torch.rand(5, generator=g)
        un.copy_(u)
        graph.replay()
        want, _, margin = ref.sample(x.cpu(), u, **kw)
        assert min(margin) > 2.0 ** -30 and token.tolist() == want


def test_no_rows_launch_nothing(dev):  # noqa: F811
    before = m.launch_count()
    m.lora_sample(torch.empty(0, dtype=torch.int32, device=dev), torch.empty((0, 50), device=dev), torch.empty(0, device=dev))
    assert m.launch_count() == before


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows_of_a_large_vocabulary(dev, dtype):  # noqa: F811
    """Rows that are read again instead of held, at odd addresses: peaked, flat, of few values, of one value, of -inf, with
    each of the limits and none."""
    rows, vocab = 160, 128001
    g = torch.Generator(device=dev).manual_seed(17)
    wide = torch.empty((rows, vocab + 5), device=dev).normal_(0, 2.5, generator=g)
    wide[:, 1000:1040] += 10
    wide[5::10] *= 0.01
    wide[6::10] = wide[6::10].round()
    wide[7::20] = 1.25
    wide[8::20, 3:] = float("-inf")
    wide[9::20] *= 40
    wide[3, :] = float("-inf")
    x = wide.to(dtype)[:, 3:vocab + 3]
    c = torch.Generator().manual_seed(18)
    u, kw = torch.rand(rows, generator=c), limits(rows, vocab, c)
    kw["top_k"][::3] = kw["top_k"][::3].clamp(max=60)
    kw["temperature"][::11] = 0
    token, lp = torch.empty(rows, dtype=torch.int32, device=dev), torch.empty(rows, device=dev)
    m.lora_sample(token, x, u.to(dev), logprob=lp, **{k: v.to(dev) for k, v in kw.items()})
    want, want_lp, margin = ref.sample(x, u, **kw)
    bad = [i for i in range(rows) if int(token[i]) != want[i] and margin[i] > 2.0 ** -30]
    assert not bad and sum(t > 2.0 ** -30 for t in margin) > rows - 5, (bad, [want[i] for i in bad], token[bad].tolist())
    near = torch.tensor(want_lp)
    fine = torch.isfinite(near)
    assert ((lp.cpu().double() - near).abs()[fine] <= 12 * ref.U * (1 + near.abs()[fine])).all()
