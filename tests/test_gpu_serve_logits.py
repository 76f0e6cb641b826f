"""lora_logits_adjust against the definition in 64 bits (serve_ref.logits, with its derived tolerance)."""
import pytest
import torch

import adapter_gemv_gb300 as m
import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import os
    if not os.path.exists(m.LIB_PATH):
        from adapter_gemv_gb300 import build
        build.build()
    return torch.device("cuda:0")


def make(rows, vocab, dtype, history, biases, requests=None, seed=0):
    g = torch.Generator().manual_seed(seed + vocab)
    n = requests or rows
    r = lambda lo, hi: torch.empty(n).uniform_(lo, hi, generator=g)  # noqa: E731
    x = torch.empty((rows, vocab)).normal_(0, 3, generator=g).to(dtype)
    x[:, ::17] = 0
    tokens = (torch.rand((n, max(history, 1)), generator=g) ** 3 * vocab).to(torch.int32)
    total = torch.randint(0, history + 1, (n,), generator=g).to(torch.int32)
    total[0] = history
    prompt = (total * torch.rand(n, generator=g)).to(torch.int32)
    count = torch.randint(0, biases + 1, (n,), generator=g)
    off = torch.cat([torch.zeros(1), count.cumsum(0)]).to(torch.int32)
    k = int(off[-1])
    tok = torch.randint(0, vocab, (k,), generator=g).to(torch.int32)
    if k > 2:
        tok[1] = tok[0]  # one id twice: the last entry counts
    mask = torch.randint(-2 ** 31, 2 ** 31, (3, (vocab + 31) // 32 + 1), generator=g).to(torch.int32)
    return dict(x=x, request=None, tokens=tokens, prompt_len=prompt, total_len=total, repetition=r(0.8, 1.4),
                presence=r(-1, 1), frequency=r(-0.3, 0.6), temperature=r(0.2, 2), bias=(off, tok, torch.randn(k, generator=g)),
                mask=mask, mask_index=torch.randint(-1, 3, (n,), generator=g).to(torch.int32))


NAMES = ("tokens", "prompt_len", "total_len", "repetition", "presence", "frequency", "temperature", "mask", "mask_index")


def run(a, dev, in_place=False, pad=0, out_pad=None, status=None):
    rows, vocab = a["x"].shape
    wide = torch.full((rows, vocab + pad), 55.0, dtype=a["x"].dtype, device=dev)
    wide[:, :vocab] = a["x"].to(dev)
    x = wide[:, :vocab]
    out_wide = torch.full((rows, vocab + (pad if out_pad is None else out_pad)), 55.0, dtype=a["x"].dtype, device=dev)
    out = x if in_place else out_wide[:, :vocab]
    kw = {k: None if a[k] is None else a[k].to(dev) for k in NAMES}
    if a["bias"] is not None:
        kw["bias"] = tuple(t.to(dev) for t in a["bias"])
    if a["request"] is not None:
        kw["row_request"] = a["request"].to(dev)
    m.lora_logits_adjust(out, x, status=status, **kw)
    torch.cuda.synchronize()
    for w in (wide, out_wide):
        assert (w[:, vocab:] == 55).all()
    if not in_place:
        assert torch.equal(x.cpu().nan_to_num(123.0), a["x"].nan_to_num(123.0))
    return out.cpu()


def check(a, got):
    want, tol = ref.logits(**a)
    ref.assert_within(got, want, tol, "logits")


@pytest.mark.parametrize("rows, vocab, history, biases", [
    (1, 1, 3, 1), (1, 31, 0, 0), (3, 33, 50, 4), (2, 1000, 300, 9), (2, 4097, 2000, 40), (1, 8191, 77, 3), (5, 2048, 4, 300),
    (1, 32000, 700, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pads", [(0, None), (5, 2)])
def test_logits(dev, rows, vocab, history, biases, dtype, pads):
    a = make(rows, vocab, dtype, history, biases)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = run(a, dev, pad=pads[0], out_pad=pads[1], status=st)
    assert int(st.item()) == 0
    check(a, got)
    assert torch.equal(run(a, dev, in_place=True, pad=pads[0]), got)


@pytest.mark.parametrize("without", ["history", "repetition", "presence", "frequency", "temperature", "bias", "mask", "all"])
def test_parts_left_out(dev, without):
    a = make(3, 5001, torch.float32, 60, 5)
    drop = {"history": ("tokens", "prompt_len", "total_len"), "mask": ("mask", "mask_index"),
            "all": NAMES + ("bias",)}.get(without, (without,))
    for k in drop:
        a[k] = None
    got = run(a, dev)
    check(a, got)
    if without == "all":
        assert torch.equal(got, a["x"])


def test_rows_of_requests_and_padding(dev):
    a = make(4, 3001, torch.float32, 40, 5, requests=7)
    a["request"] = torch.tensor([6, -1, 0, 6], dtype=torch.int32)
    got = run(a, dev)
    assert (got[1] == 55).all()
    got[1] = a["x"][1]
    check(a, got)


def test_masked_infinities_and_nan(dev):
    a = make(2, 2500, torch.float32, 30, 3)
    a["mask_index"][:] = 0
    barred = [t for t in range(2500) if not (int(a["mask"][0, t // 32]) >> (t % 32)) & 1]
    a["x"][0, barred] = float("nan")
    a["x"][1, barred[:50]] = float("inf")
    a["x"][1, barred[50:99]] = torch.finfo(torch.float32).min
    got = run(a, dev)
    assert torch.isneginf(got[:, barred]).all()
    check(a, got)
    a["mask"][:] = 0  # a grammar that allows nothing
    assert torch.isneginf(run(a, dev)).all()
    a["mask_index"][:] = -1
    a["x"][1, 5], a["x"][1, 6] = float("-inf"), torch.finfo(torch.float32).min
    got = run(a, dev)
    assert torch.isneginf(got[1, 5]) and torch.isnan(got[0, barred]).all()


def test_temperature_zero_leaves_the_scale(dev):
    a = make(2, 600, torch.float32, 30, 3)
    a["temperature"][:] = torch.tensor([0.0, 0.5])
    check(a, run(a, dev))


def test_bad_entries_and_rows(dev):
    a = make(5, 900, torch.float32, 30, 6)
    a["total_len"][:] = 30
    a["prompt_len"][:] = 3
    a["tokens"][1, 4], a["tokens"][1, 29] = -1, 900
    k = int(a["bias"][0][1])
    if k:
        a["bias"][1][0] = 1 << 30
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = run(a, dev, status=st)
    assert int(st.item()) == m.STATUS_BAD_TOKEN
    check(a, got)
    for name, at, value, bit in (("total_len", 1, 31, 64), ("total_len", 2, -1, 64), ("prompt_len", 0, 31, 64),
                                 ("prompt_len", 3, -1, 64), ("mask_index", 4, 3, 2), ("mask_index", 4, -2, 2)):
        b = make(5, 900, torch.float32, 30, 6)
        b[name][at] = value
        st.zero_()
        got = run(b, dev, status=st)
        assert int(st.item()) == bit and (got[at] == 55).all(), name
        b[name][at] = 0 if name != "mask_index" else -1
        keep = [i for i in range(5) if i != at]
        want, tol = ref.logits(**b)
        ref.assert_within(got[keep], want[keep], tol[keep], name)
    b = make(5, 900, torch.float32, 30, 6)
    b["bias"][0][3] = b["bias"][0][-1] + 1
    st.zero_()
    got = run(b, dev, status=st)
    assert int(st.item()) == m.STATUS_BAD_LENGTH and (got[2:4] == 55).all()
    b = make(3, 900, torch.float32, 30, 6)
    b["request"] = torch.tensor([0, 3, -2], dtype=torch.int32)
    st.zero_()
    got = run(b, dev, status=st)
    assert int(st.item()) == m.STATUS_BAD_REQUEST and (got[1:] == 55).all()


def test_many_rows(dev):
    """More rows than a grid dimension holds."""
    x = torch.randn((70001, 9), device=dev)
    temp = torch.rand(70001, device=dev) + 0.5
    out = torch.empty_like(x)
    m.lora_logits_adjust(out, x, temperature=temp)
    assert torch.equal(out, x / temp[:, None])


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("history, biases", [(33000, 5), (50, 70000), (33000, 140000), (32767, 65535)])
def test_long_histories_and_lists(dev, rows, history, biases):
    """Counts beyond 16 bits, and lists whose entry numbers are; many rows take the larger slices."""
    a = make(2, 3001, torch.float32, history, biases)
    a["total_len"][:] = history
    a["tokens"][1, :] = 7  # one token all the way
    a["prompt_len"][1] = 3
    a["bias"] = (torch.tensor([0, biases, biases], dtype=torch.int32), torch.randint(0, 3001, (biases,)).to(torch.int32),
                 torch.randn(biases))
    want, tol = ref.logits(**a)
    a["request"] = torch.arange(2, dtype=torch.int32).repeat(rows)
    a["x"] = a["x"].repeat(rows, 1)
    got = run(a, dev)
    ref.assert_within(got, want.repeat(rows, 1), tol.repeat(rows, 1), "logits")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_batch_over_an_odd_vocabulary(dev, dtype):
    a = make(3, 40001, dtype, 900, 30)
    want, tol = ref.logits(**a)
    a["request"] = torch.arange(3, dtype=torch.int32).repeat(40)
    a["x"] = a["x"].repeat(40, 1)
    for in_place in (False, True):
        ref.assert_within(run(a, dev, in_place=in_place, pad=3), want.repeat(40, 1), tol.repeat(40, 1), "logits")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_temperatures_of_all_sizes(dev, dtype):
    """Quotients at both ends of the range, infinities and zeros among the logits: what a division gives."""
    temp = torch.tensor([1e-38, 1e-30, 1e-3, 0.1, 1 / 3, 1.0, 1.9999999, 3.0, 1e10, 1e30, 3e38, 2.0 ** -100, 1e-42], device=dev)
    x = torch.randn((13, 5000), device=dev)
    x[:, :8] = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), 3e38, -3e38, 1e-38, 65504.0], device=dev)
    x = x.to(dtype)
    out = torch.empty_like(x)
    m.lora_logits_adjust(out, x, temperature=temp)
    want = (x.double() / temp.double()[:, None]).float().to(dtype)
    tiny = want.float().abs() < 1e-37  # (rounded again below the normal numbers)
    assert torch.equal(out[~tiny], want[~tiny])
    assert ((out.double() - want.double()).abs()[tiny] <= 2e-45).all() or dtype != torch.float32


@pytest.mark.parametrize("first", [0, 3, 400, 511])
@pytest.mark.parametrize("alone", [False, True])
def test_history_in_a_column_view(dev, first, alone):
    """tokens as columns of a wider matrix, up to its very end: a row's ids are the view's, and a total_len beyond them is
    an error although the matrix's rows go on."""
    history = 512 - first
    a = make(1 if alone else 5, 3001, torch.float32, history, 4)
    a["total_len"][:] = history
    a["prompt_len"][:] = history // 2
    n = a["x"].shape[0]
    wide = torch.full((7, 512), 17, dtype=torch.int32, device=dev)
    view = wide[7 - n:, first:]
    view.copy_(a["tokens"])
    kw = {k: a[k].to(dev) for k in NAMES if k != "tokens"}
    kw["bias"] = tuple(t.to(dev) for t in a["bias"])
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    x = a["x"].to(dev)
    out = torch.full_like(x, 55.0)
    m.lora_logits_adjust(out, x, tokens=view, status=st, **kw)
    assert int(st.item()) == 0
    check(a, out.cpu())
    if n > 1:  # one id more than row 1 has: the first of the next row, if the matrix's rows were taken for the view's
        kw["total_len"][1] = history + 1
        out.fill_(55.0)
        m.lora_logits_adjust(out, x, tokens=view, status=st, **kw)
        want, tol = ref.logits(**a)
        keep = [0, 2, 3, 4]
        ref.assert_within(out.cpu()[keep], want[keep], tol[keep], "logits")
        assert int(st.item()) == m.STATUS_BAD_LENGTH and (out[1] == 55).all()


def test_as_many_rows_as_are_counted(dev):
    """2^31 - 1 rows: the launches' first rows end below 2^31."""
    rows = 2 ** 31 - 1
    x = torch.arange(4096, dtype=torch.float16, device=dev).repeat((rows + 4095) // 4096)[:rows, None]
    out = torch.empty_like(x)
    m.lora_logits_adjust(out, x)
    assert torch.equal(out, x)
