"""lora_kv_attention against the definition in 64 bits (serve_ref.attention, with its derived tolerance)."""
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


class Case:
    """A cache whose tokens beyond every request's length, and whose free pages, are NaN."""

    def __init__(self, dev, lens, hq, hk, d, pt=16, heads_first=False, dtype=torch.bfloat16, window=0, per=1, layers=2,
                 seed=0, q_std=1.0, pad_cols=0, free_pages=3):
        g = torch.Generator(device=dev).manual_seed(seed + 1000 * d + hq)
        n, self.layer, self.window, self.hq = len(lens), layers - 1, window, hq
        pages = [ref.ceil(x, pt) for x in lens]
        total, width = sum(pages) + free_pages, max(pages + [1]) + 1
        shape = (layers, total, hk, pt, d) if heads_first else (layers, total, pt, hk, d)
        k, v = (torch.full(shape, float("nan"), dtype=dtype, device=dev) for _ in range(2))
        self.k, self.v = (x.transpose(2, 3) if heads_first else x for x in (k, v))
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        wide = torch.full((n, width + 3), -9, dtype=torch.int32, device=dev)
        self.table = wide[:, :width]
        at = 0
        for r, x in enumerate(lens):
            mine = ids[at:at + pages[r]]
            at += pages[r]
            self.table[r, :pages[r]] = mine
            t = torch.arange(x, device=dev)
            for c in (self.k, self.v):
                c[self.layer, mine[t // pt].long(), t % pt] = torch.empty((x, hk, d), dtype=dtype,
                                                                          device=dev).normal_(generator=g)
        pos = [x - per + j for x in lens for j in range(per)]
        self.position = torch.tensor([max(p, -1) for p in pos], dtype=torch.int32, device=dev)
        self.request = torch.arange(n, dtype=torch.int32, device=dev).repeat_interleave(per)
        rows = n * per
        qw = torch.empty((rows, hq * d + pad_cols), dtype=dtype, device=dev).normal_(0, q_std, generator=g)
        self.q = qw[:, :hq * d]
        self.out_wide = torch.full((rows, hq * d + pad_cols), 77.0, dtype=dtype, device=dev)
        self.out = self.out_wide[:, :hq * d]
        self.lse = torch.full((rows, hq), 77.0, device=dev)
        self.scale = d ** -0.5
        self.cache = m.make_kv_cache(self.k, self.v)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspace = m.kv_attention_workspace(self.cache, hq)

    def call(self, **kw):
        a = dict(row_request=self.request, lse=self.lse, scale=self.scale, window=self.window, status=self.status)
        a.update(kw)
        return m.KvAttention(self.out, self.q, self.cache, self.table, self.position, self.layer, self.workspace, **a)

    def check(self, rows=None):
        d = self.q.shape[1] // self.hq
        sel = slice(None) if rows is None else rows
        want = ref.attention(self.q.reshape(-1, self.hq, d)[sel], self.k, self.v, self.layer, self.table, self.request[sel],
                             self.position[sel], self.scale, self.window)
        ref.assert_within(self.out.reshape(-1, self.hq, d)[sel], want[0], want[2], "out")
        ref.assert_within(self.lse[sel], want[1], want[3], "lse")

    def run(self, **kw):
        self.call(**kw)()
        torch.cuda.synchronize()
        assert (self.out_wide[:, self.out.shape[1]:] == 77).all()


LENS = [1, 2, 15, 16, 17, 31, 33, 100, 257]
SHAPES = [
    # lens, hq, hk, d, page_tokens, heads_first, dtype
    ([1], 1, 1, 8, 16, False, torch.bfloat16),
    ([61], 32, 32, 128, 16, False, torch.bfloat16),
    (LENS, 4, 4, 128, 16, False, torch.bfloat16),
    (LENS, 8, 1, 128, 32, True, torch.float16),
    (LENS, 16, 2, 64, 16, True, torch.bfloat16),
    (LENS, 15, 5, 80, 24, False, torch.float16),
    (LENS, 32, 2, 128, 64, False, torch.bfloat16),
    (LENS, 24, 2, 256, 8, True, torch.bfloat16),
    (LENS, 40, 2, 96, 16, False, torch.float16),
    (LENS, 34, 1, 64, 16, False, torch.bfloat16),
    (LENS, 6, 6, 256, 128, False, torch.float16),
    (LENS, 7, 1, 16, 1, False, torch.bfloat16),
    (LENS, 14, 2, 72, 3, True, torch.float16),
    (LENS, 9, 3, 40, 1000, False, torch.bfloat16),
    (LENS, 2, 2, 248, 5, False, torch.bfloat16),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window, per", [(0, 1), (20, 1), (0, 3), (1, 2)])
def test_attention(dev, shape, window, per):
    lens, hq, hk, d, pt, heads_first, dt = shape
    c = Case(dev, lens, hq, hk, d, pt, heads_first, dt, window, per, pad_cols=8)
    c.run()
    assert int(c.status.item()) == 0
    c.check()


@pytest.mark.parametrize("lens, hq, hk, d, dtype", [
    ([5000], 8, 1, 128, torch.bfloat16), ([5000], 32, 32, 128, torch.float16), ([40001], 64, 8, 128, torch.bfloat16),
    ([3, 20000, 1, 700], 16, 1, 64, torch.bfloat16), ([9000, 1, 1, 9001], 12, 1, 256, torch.float16),
    ([70000], 1, 1, 128, torch.bfloat16), ([17] * 700, 4, 2, 128, torch.bfloat16),
    ([300 + 13 * i for i in range(64)], 64, 8, 128, torch.bfloat16)])
def test_attention_long_and_many(dev, lens, hq, hk, d, dtype):
    """Rows split over the GPU, and more rows than its processors."""
    c = Case(dev, lens, hq, hk, d, 32, True, dtype)
    c.run()
    assert int(c.status.item()) == 0
    c.check()


def test_more_rows_than_a_launch(dev):
    n = 5003
    c = Case(dev, [1 + (7 * i) % 19 for i in range(n)], 2, 1, 64, 16)
    c.run()
    c.check()


def test_empty_rows_and_default_rows(dev):
    """position -1 sees nothing: 0 and -inf; without row_request row i is request i; without lse none is written."""
    c = Case(dev, [40, 0, 7, 0, 0, 300], 8, 2, 64)
    assert c.position.tolist() == [39, -1, 6, -1, -1, 299]
    c.run()
    c.check()
    assert (c.out[c.position < 0] == 0).all() and torch.isneginf(c.lse[c.position < 0]).all()
    first = c.out.clone()
    c.lse.fill_(5)
    c.run(row_request=None, lse=None)
    assert torch.equal(c.out, first) and (c.lse == 5).all()
    c.position.fill_(-1)
    c.run()
    assert (c.out == 0).all() and torch.isneginf(c.lse).all()


@pytest.mark.parametrize("hq, hk, d", [(8, 8, 128), (16, 2, 64), (24, 2, 128)])
def test_values_that_exponentials_overflow_on(dev, hq, hk, d):
    """Scores of hundreds, of both signs: the weights go to single tokens."""
    c = Case(dev, [3, 50, 1000], hq, hk, d, q_std=60.0)
    c.run()
    c.check()


def test_infinite_scores_stay_where_they_are(dev):
    """An infinite key makes its own request's rows NaN (inf - inf) or follows the softmax's limit; the others' do not
    change."""
    c = Case(dev, [50, 60], 4, 2, 64)
    c.run()
    clean = c.out.clone()
    page, t = int(c.table[0, 1]), 3
    c.k[c.layer, page, t, 0, 5] = float("inf")
    c.run()
    assert torch.equal(c.out[1], clean[1])
    assert torch.equal(c.out[0, 128:], clean[0, 128:])  # the other key-value head
    # masked by a window that starts behind it
    c.window = 20
    c.run()
    assert torch.isfinite(c.out).all()
    c.check()


def test_bad_rows_and_pages(dev):
    c = Case(dev, [40, 50, 60, 70, 100], 8, 2, 64)
    c.request[1], c.request[2] = 5, -1
    c.position[3] = c.table.shape[1] * 16
    c.run()
    assert int(c.status.item()) == m.STATUS_BAD_REQUEST | m.STATUS_BAD_LENGTH
    assert (c.out[1:4] == 77).all() and (c.lse[1:4] == 77).all()
    c.check([0, 4])
    c.position[3] = -2
    c.status.zero_()
    c.run()
    assert int(c.status.item()) == m.STATUS_BAD_REQUEST | m.STATUS_BAD_LENGTH and (c.out[3] == 77).all()
    # pages that do not exist: their tokens are not seen
    c.status.zero_()
    c.table[4, 2], c.table[4, 4], c.table[0, 0] = -1, c.k.shape[1], 1 << 30
    c.run()
    assert int(c.status.item()) & m.STATUS_BAD_PAGE
    c.check([0, 4])
    c.table[0, :3] = -5
    c.run()
    assert (c.out[0] == 0).all() and torch.isneginf(c.lse[0]).all()


def test_same_bits_again_and_workspace_left_clean(dev):
    """Calls of several shapes share a workspace in turn; each gives the bits it gave before."""
    cases = [Case(dev, [4000, 30], 8, 1, 128), Case(dev, [1] * 40, 8, 8, 128), Case(dev, [900, 10, 12000], 16, 1, 128),
             Case(dev, [77], 32, 32, 128)]
    ws = m.kv_attention_workspace(cases[0].cache, 32)
    calls = []
    for c in cases:
        c.workspace = ws
        calls.append(c.call())
        calls[-1]()
    first = [(c.out.clone(), c.lse.clone()) for c in cases]
    for _ in range(3):
        for i in (2, 0, 3, 1, 0, 2):
            cases[i].out.fill_(0)
            calls[i]()
            assert torch.equal(cases[i].out, first[i][0]) and torch.equal(cases[i].lse, first[i][1])
    for c in cases:
        c.check()


def test_another_stream_and_graph_replay(dev):
    """On a stream of its own; captured, replayed with other lengths in the same buffers."""
    c = Case(dev, [500, 33, 800], 16, 2, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = c.call()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for pos in ([499, 32, 799], [3, 20, 700], [-1, 0, 799]):
        c.position.copy_(torch.tensor(pos, dtype=torch.int32))
        c.out.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_offsets_beyond_32_bits(dev):
    """A cache of more than 2^31 elements (and 2^32 bytes) each for K and V, a request's pages at its far end."""
    pt, hk, d = 16, 8, 128
    pages = (1 << 31) // (pt * hk * d) + 40
    k, v = (torch.empty((1, pages, pt, hk, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    n, g = 30, torch.Generator(device=dev).manual_seed(1)
    for x in (k, v):
        x[0, -n:].normal_(generator=g)
    c = Case(dev, [n * pt - 3], 64, hk, d)
    c.k, c.v, c.cache, c.layer = k, v, m.make_kv_cache(k, v), 0
    c.table[0, :n] = torch.arange(pages - n, pages, dtype=torch.int32)
    c.run()
    c.check()
    slot = torch.tensor([pages * pt - 1], device=dev)
    row = torch.ones((1, hk * d), dtype=torch.bfloat16, device=dev)
    m.lora_kv_append(c.cache, row, row * 2, slot, 0)
    assert (k[0, -1, -1] == 1).all() and (v[0, -1, -1] == 2).all()


def test_cache_in_the_adapters_page_pool(dev):
    """The cache as a view of an S-LoRA style page pool: a page of 4096 elements holds K and V of 8 tokens."""
    pool = torch.full((60, 4096), float("nan"), dtype=torch.bfloat16, device=dev)
    hk, d, pt = 2, 128, 8
    kv = pool.view(60, 2, pt, hk, d)
    c = Case(dev, [100, 21], 8, hk, d, pt)
    k, v = kv[:, 0][None], kv[:, 1][None]
    for r, x in enumerate((100, 21)):
        t = torch.arange(x, device=dev)
        for dst, src in ((k, c.k), (v, c.v)):
            dst[0, c.table[r, t // pt].long(), t % pt] = src[c.layer, c.table[r, t // pt].long(), t % pt]
    c.k, c.v, c.cache, c.layer = k, v, m.make_kv_cache(k, v), 0
    c.run()
    c.check()


def with_rows(c, rows, g):
    """The case's requests with other rows: (request, position) pairs."""
    dev, hq, d = c.q.device, c.hq, c.q.shape[1] // c.hq
    c.request = torch.tensor([r for r, _ in rows], dtype=torch.int32, device=dev)
    c.position = torch.tensor([p for _, p in rows], dtype=torch.int32, device=dev)
    c.q = torch.empty((len(rows), hq * d), dtype=c.q.dtype, device=dev).normal_(generator=g)
    c.out_wide = c.out = torch.full((len(rows), hq * d), 77.0, dtype=c.q.dtype, device=dev)
    c.lse = torch.full((len(rows), hq), 77.0, device=dev)
    return c


@pytest.mark.parametrize("hq, hk, d, pt, dtype", [
    (1, 1, 64, 16, torch.bfloat16), (8, 8, 128, 16, torch.float16), (15, 5, 80, 24, torch.float16),
    (32, 8, 128, 32, torch.bfloat16), (8, 1, 128, 16, torch.bfloat16), (12, 1, 64, 8, torch.bfloat16),
    (10, 2, 256, 16, torch.float16), (40, 2, 64, 16, torch.bfloat16)])
@pytest.mark.parametrize("window", [0, 1, 30, 400])
@pytest.mark.parametrize("least", [0, 1100, 2600])
def test_rows_of_one_request_share_its_tiles(dev, hq, hk, d, pt, dtype, window, least):
    """Prompts, drafted continuations, rows that repeat, go backwards, skip, see nothing or have other requests'
    rows between them: whatever rows are taken together, each sees its own tokens only."""
    import random
    rnd = random.Random(hq * d + window)
    lens = [1, 5, 40, 300, 1000, 17, 64]
    c = Case(dev, lens, hq, hk, d, pt, dtype=dtype, window=window, layers=1)
    rows = [(2, p) for p in range(40)]  # a prompt
    rows += [(3, p) for p in (295, 296, 297, 298, 299)]  # drafted tokens
    rows += [(4, 999), (4, 500), (4, 501), (4, 501), (4, 20), (4, 999)]  # gaps, repeats, backwards
    rows += [(0, 0), (1, 4), (0, 0), (1, 3), (5, 16), (5, -1), (5, 15), (5, 14), (6, 63), (6, 62), (6, 0)]
    while len(rows) < 150 or len(rows) * hk < least:
        r = rnd.randrange(7)
        p = rnd.randrange(lens[r])
        rows += [(r, min(p + k, lens[r] - 1)) for k in range(rnd.choice((1, 1, 2, 3, 9, 18)))]
    with_rows(c, rows, torch.Generator(device=dev).manual_seed(5))
    c.run()
    assert int(c.status.item()) == 0
    c.check()
    first = c.out.clone()
    c.run()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("more", [0, 300])
def test_bad_rows_among_packed_ones(dev, more):
    c = Case(dev, [100, 200], 4, 4, 64, layers=1)
    rows = [(0, 97), (0, 98), (0, 99), (0, 10 ** 6), (0, 99), (2, 5), (1, 198), (1, 199), (-1, 3), (1, 199), (1, -2), (1, 7)]
    rows += [(k % 30 // 15, 40 + k % 15) for k in range(more)]
    with_rows(c, rows, torch.Generator(device=dev).manual_seed(6))
    c.run()
    assert int(c.status.item()) == m.STATUS_BAD_REQUEST | m.STATUS_BAD_LENGTH
    bad = [3, 5, 8, 10]
    assert (c.out[bad] == 77).all() and (c.lse[bad] == 77).all()
    c.check([i for i in range(len(rows)) if i not in bad])
    # a page that is gone behind every row's window is not looked at
    c.window = 20
    rows = [(0, 30), (0, 99), (0, 98), (1, 150), (1, 151)]
    rows += [(1, 150 + k % 15) for k in range(more)]
    with_rows(c, rows, torch.Generator(device=dev).manual_seed(7))
    c.table[0, 3], c.table[1, 0] = -1, -1
    c.status.zero_()
    c.run()
    assert int(c.status.item()) == 0
    c.check()


def test_a_long_prompt_in_pieces_of_many_rows(dev):
    """2000 rows of one request, more than a launch's, and 3 others."""
    c = Case(dev, [2100, 50, 3], 8, 2, 128, layers=1)
    rows = [(0, p) for p in range(100, 2100)] + [(1, 49), (2, 2), (2, 1)]
    with_rows(c, rows, torch.Generator(device=dev).manual_seed(8))
    c.run()
    c.check()


@pytest.mark.parametrize("hq, hk, d, pt, dtype", [
    (4, 2, 128, 16, torch.bfloat16), (15, 5, 80, 24, torch.float16), (32, 16, 64, 16, torch.float16),
    (32, 16, 128, 8, torch.bfloat16), (16, 16, 256, 16, torch.bfloat16), (128, 16, 128, 16, torch.float16)])
@pytest.mark.parametrize("window", [0, 37])
def test_a_value_that_only_later_rows_see(dev, hq, hk, d, pt, dtype, window):
    """Infinities and NaN in a token's V reach the rows that see it, at those elements, and no other."""
    c = Case(dev, [260, 90], hq, hk, d, pt, dtype=dtype, window=window, layers=1)
    rows = [(0, p) for p in range(60, 260)] + [(1, p) for p in range(70, 90)]
    with_rows(c, rows, torch.Generator(device=dev).manual_seed(9))
    wild = {(0, 100): (float("inf"), [0, d - 1]), (0, 163): (float("nan"), [5]), (0, 164): (float("-inf"), [d // 2]),
            (0, 259): (float("nan"), list(range(d))), (1, 80): (float("inf"), [1])}
    for (r, t), (x, els) in wild.items():
        c.v[c.layer, int(c.table[r, t // pt]), t % pt, :, els] = x
    c.run()
    assert int(c.status.item()) == 0
    out = c.out.reshape(-1, hq, d)
    for (r, t), (x, els) in wild.items():
        c.v[c.layer, int(c.table[r, t // pt]), t % pt, :, els] = 0
    want, lse, tol, ltol = ref.attention(c.q.reshape(-1, hq, d), c.k, c.v, c.layer, c.table, c.request, c.position, c.scale,
                                         window)
    ref.assert_within(c.lse, lse, ltol, "lse")
    hit = torch.zeros((len(rows), d), dtype=torch.bool, device=dev)
    for i, (r, p) in enumerate(rows):
        for (wr, t), (_, els) in wild.items():
            if wr == r and (max(0, p + 1 - window) if window else 0) <= t <= p:
                hit[i, els] = True
    hit = hit[:, None, :].expand(-1, hq, -1)
    assert not torch.isfinite(out[hit]).any()
    ref.assert_within(out[~hit], want[~hit], tol[~hit], "out")


@pytest.mark.parametrize("lens, per, hq, hk, d", [([5, 9000, 40], 1, 8, 1, 128), ([300] * 40, 3, 15, 5, 80), ([70], 1, 40, 2, 64)])
def test_in_place(dev, lens, per, hq, hk, d):
    """out may be q: rows that are whole, split over the GPU, share tiles, or have more heads than a tile."""
    c = Case(dev, lens, hq, hk, d, per=per)
    c.run()
    want = c.out.clone()
    q = c.q.clone()
    call = m.KvAttention(q, q, c.cache, c.table, c.position, c.layer, c.workspace, row_request=c.request, lse=c.lse,
                         scale=c.scale)
    call()
    assert torch.equal(q, want)


@pytest.mark.parametrize("hq, hk, d", [(8, 8, 128), (15, 5, 80), (64, 16, 64), (16, 2, 256), (40, 2, 64)])
@pytest.mark.parametrize("rows_per_request", [0, 1, 2, 3, 7, 2 ** 31 - 1])
def test_rows_per_request_changes_no_result(dev, hq, hk, d, rows_per_request):
    """Right or wrong, a request's number of rows decides what shares a tile only: drafts of 1 to 6 rows and padding in a
    table with more places than requests, few rows and many."""
    lens = [300, 17, 64, 1, 150]
    for times in (1, 40):
        c = Case(dev, lens + [5] * 300, hq, hk, d, layers=1)
        rows = []
        for r, n in enumerate(lens):
            rows += [(r, p) for p in range(max(0, n - r - 2), n)]
        with_rows(c, (rows + [(-1, -1)] * 9) * times, torch.Generator(device=dev).manual_seed(13))
        c.run(rows_per_request=rows_per_request)
        assert int(c.status.item()) == 0
        c.check()
