"""lora_kv_layout and lora_kv_append against the plain implementations of serve_ref: whole numbers equal,
rotated values within the derived tolerance, everything else bit for bit."""
import random

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


OUT = ("row_request", "position", "cache_slot", "row_slot", "seg_offsets", "seg_slot", "kv_len_out", "free_state_out",
       "page_table", "free_ring")


def layout_case(seed, requests, page_tokens, max_new, padding, leave=0.1, extra_pages=7, longest=200):
    rnd = random.Random(seed)
    lens = [rnd.choice([0, 1, rnd.randint(0, longest), page_tokens * rnd.randint(0, 4)]) for _ in range(requests)]
    new = [-1 if rnd.random() < leave else rnd.choice([0, 1, 1, rnd.randint(0, max_new)]) for _ in range(requests)]
    max_pages = max([ref.ceil(a + max(b, 0), page_tokens) for a, b in zip(lens, new)] + [1]) + 1
    used = sum(ref.ceil(a, page_tokens) for a in lens)
    need = sum(ref.ceil(a + b, page_tokens) - ref.ceil(a, page_tokens) for a, b in zip(lens, new) if b >= 0)
    pages = used + need + extra_pages
    ids = list(range(pages))
    rnd.shuffle(ids)
    table, at = [], 0
    for a in lens:
        k = ref.ceil(a, page_tokens)
        table.append(ids[at:at + k] + [-1] * (max_pages - k))
        at += k
    head, count = rnd.randrange(pages), pages - used
    ring = [-1] * pages
    for i in range(count):
        ring[(head + i) % pages] = ids[used + i]
    rows = sum(max(b, 0) for b in new) + padding
    return dict(new_tokens=new, kv_len=lens, page_table=table, ring=ring, state=[head, count], page_tokens=page_tokens,
                num_rows=rows, adapter_slot=[rnd.randint(-1, 9) for _ in range(requests)])


def run_layout(case, dev, alias=False, stride_pad=0, status=None):
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    width = len(case["page_table"][0]) if case["page_table"] else 4
    wide = torch.full((max(1, len(case["page_table"])), width + stride_pad), -7, dtype=torch.int32, device=dev)
    table = wide[:len(case["page_table"]), :width]
    if case["page_table"]:
        table.copy_(t(case["page_table"]))
    kv_len, state = t(case["kv_len"]), t(case["state"])
    b = m.KvBatch(t(case["new_tokens"]), kv_len, table, t(case["ring"]), state, case["page_tokens"], case["num_rows"],
                  adapter_slot=None if case["adapter_slot"] is None else t(case["adapter_slot"]),
                  kv_len_out=kv_len if alias else torch.empty_like(kv_len),
                  free_state_out=state if alias else torch.empty_like(state))
    m.lora_kv_layout(b, status)
    torch.cuda.synchronize()
    if stride_pad:
        assert (wide[:, width:] == -7).all()
    return b


def check_layout(case, b, status=None):
    want = ref.layout(**case)
    for k in OUT:
        got = getattr(b, k).tolist()
        assert got == want[k], k
    if status is not None:
        assert int(status.item()) == want["status"]
    return want


@pytest.mark.parametrize("requests, page_tokens, max_new, padding", [
    (1, 16, 1, 0), (1, 1, 40, 3), (3, 16, 100, 0), (32, 16, 1, 0), (37, 24, 50, 11), (257, 8, 3, 1), (1000, 16, 30, 100),
    (1025, 32, 2, 0), (4096, 16, 4, 5), (m.KV_MAX_REQUESTS, 7, 3, 9)])
@pytest.mark.parametrize("alias", [False, True])
def test_layout(dev, requests, page_tokens, max_new, padding, alias):
    case = layout_case(requests * 31 + page_tokens, requests, page_tokens, max_new, padding)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    b = run_layout(case, dev, alias, stride_pad=5, status=st)
    assert check_layout(case, b, st)["status"] == 0


def test_layout_no_requests_no_rows_no_adapters(dev):
    case = dict(new_tokens=[], kv_len=[], page_table=[], ring=[4, 5], state=[1, 2], page_tokens=16, num_rows=5,
                adapter_slot=None)
    check_layout(case, run_layout(case, dev))
    case = dict(layout_case(5, 9, 16, 0, 0), adapter_slot=None)
    case["new_tokens"] = [min(b, 0) for b in case["new_tokens"]]
    case["num_rows"] = 0
    check_layout(case, run_layout(case, dev))


def test_layout_all_pages_taken_and_ring_full(dev):
    # the last free page is taken, and every page given back
    case = layout_case(11, 20, 16, 60, 0, leave=0.0, extra_pages=0)
    assert check_layout(case, run_layout(case, dev))["free_state_out"][1] == 0
    case = layout_case(12, 20, 16, 60, 2)
    case["new_tokens"] = [-1] * 20
    assert check_layout(case, run_layout(case, dev))["free_state_out"][1] == len(case["ring"])


@pytest.mark.parametrize("what, bit", [("pages", 32), ("rows", 64), ("length", 64), ("new", 64), ("negative", 64),
                                       ("head", 64), ("count", 64), ("overfull", 64)])
@pytest.mark.parametrize("alias", [False, True])
def test_layout_errors_change_nothing(dev, what, bit, alias):
    case = layout_case(77, 40, 16, 30, 4, leave=0.2 if what == "overfull" else 0.0)
    if what == "pages":
        case["state"][1] = 1
        case["new_tokens"] = [17] * 40
        case["num_rows"] = 700
        case["page_table"] = [r + [-1, -1] for r in case["page_table"]]
    elif what == "rows":
        case["num_rows"] = sum(case["new_tokens"]) - 1
    elif what == "length":
        case["new_tokens"][3] = len(case["page_table"][0]) * 16 + 1
    elif what == "new":
        case["new_tokens"][39] = -2
    elif what == "negative":
        case["kv_len"][0] = -1
    elif what == "head":
        case["state"][0] = len(case["ring"])
    elif what == "count":
        case["state"][1] = len(case["ring"]) + 1
    else:  # more pages come back than the ring can hold
        case["state"][1] = len(case["ring"])
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    want = check_layout(case, run_layout(case, dev, alias, status=st), st)
    assert want["status"] == bit and set(want["cache_slot"]) == {-1}


def test_layout_bad_page_id_marks_its_rows(dev):
    case = layout_case(21, 12, 16, 5, 3, leave=0.0)
    r = next(i for i, (a, b) in enumerate(zip(case["kv_len"], case["new_tokens"])) if a % 16 and b > 0)
    case["page_table"][r][case["kv_len"][r] // 16] = len(case["ring"])
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    assert check_layout(case, run_layout(case, dev, status=st), st)["status"] == 8


# ---- append --------------------------------------------------------------------------------------


def make_cache(dev, dtype, layers, pages, pt, heads, d, heads_first, g):
    shape = (layers, pages, heads, pt, d) if heads_first else (layers, pages, pt, heads, d)
    k, v = (torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g) for _ in range(2))
    return (k.transpose(2, 3), v.transpose(2, 3)) if heads_first else (k, v)


APPENDS = [
    # rows, hq, hk, d, rotary, interleaved, page_tokens, heads_first, dtype
    (1, 32, 32, 128, 128, False, 16, False, torch.bfloat16),
    (5, 8, 2, 64, 64, False, 1, True, torch.float16),
    (33, 15, 5, 80, 48, False, 24, False, torch.float16),
    (7, 4, 4, 256, 256, True, 8, True, torch.bfloat16),
    (19, 6, 1, 72, 16, True, 7, False, torch.bfloat16),
    (300, 3, 3, 8, 0, False, 16, False, torch.float16),
    (4, 0, 8, 128, 128, False, 16, False, torch.bfloat16),
]


@pytest.mark.parametrize("case", APPENDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_append(dev, case, in_place):
    rows, hq, hk, d, rot, inter, pt, heads_first, dt = case
    g = torch.Generator(device=dev).manual_seed(rows * 7 + d)
    pages, layers, layer, top = ref.ceil(rows + 5, pt) + 2, 3, 1, 500
    k_cache, v_cache = make_cache(dev, dt, layers, pages, pt, hk, d, heads_first, g)
    width = (hq + 2 * hk) * d
    wide = torch.empty((rows, width + 24), dtype=dt, device=dev).normal_(generator=g)
    q, k, v = wide[:, :hq * d], wide[:, hq * d:(hq + hk) * d], wide[:, (hq + hk) * d:width]
    slot = torch.randperm(pages * pt, generator=g, device=dev)[:rows]
    skipped = torch.rand(rows, generator=g, device=dev) < 0.2
    slot = torch.where(skipped, -1, slot) if rows > 1 else slot
    position = torch.randint(0, top, (rows,), generator=g, device=dev, dtype=torch.int32)
    position = torch.where(slot < 0, -1, position).to(torch.int32)
    rope = None
    if rot:
        cos, sin = (torch.empty((top, rot // 2), device=dev).normal_(generator=g) for _ in range(2))
        rope = m.Rope(cos, sin, inter)
    q_out = q if in_place else torch.empty((rows, hq * d), dtype=dt, device=dev).normal_(generator=g)
    before = dict(wide=wide.clone(), k=k_cache.clone(), v=v_cache.clone(), q_out=q_out.clone())
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    m.lora_kv_append(m.make_kv_cache(k_cache, v_cache), k, v, slot, layer, q=q if hq else None, q_out=q_out if hq else None,
                     position=position if rot else None, rope=rope, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want_v, want_k, got_k = before["v"].clone(), before["k"].clone(), k_cache.clone()
    qb = before["wide"][:, :hq * d]
    for i in range(rows):
        s = int(slot[i])
        if s < 0:
            if hq:
                assert torch.equal(q_out[i], before["q_out"][i])
            continue
        at = (layer, s // pt, s % pt)
        want_v[at] = before["wide"][i, (hq + hk) * d:width].reshape(hk, d)
        rows_k = before["wide"][i, hq * d:(hq + hk) * d].double().reshape(hk, d)
        rows_q = qb[i].double().reshape(hq, d)
        for x, got in ((rows_k, k_cache[at]), (rows_q, q_out[i].reshape(hq, d))):
            y, mag = ref.rotate(x, int(position[i]), cos, sin, inter) if rot else (x, x.abs() * 0)
            tol = ref.rotate_tol(y, mag, dt) if rot else x * 0
            tol[:, rot:] = 0  # copied
            ref.assert_within(got, y, tol, f"row {i}")
        got_k[at] = want_k[at]
    assert torch.equal(v_cache, want_v)
    assert torch.equal(got_k, want_k)  # nothing else of the cache changed
    if not in_place:
        assert torch.equal(wide, before["wide"])
    else:
        assert torch.equal(wide[:, hq * d:], before["wide"][:, hq * d:])


def test_append_bad_rows_are_skipped_and_reported(dev):
    g = torch.Generator(device=dev).manual_seed(3)
    k_cache, v_cache = make_cache(dev, torch.bfloat16, 1, 4, 16, 2, 64, False, g)
    k, v, q = (torch.empty((6, n * 64), dtype=torch.bfloat16, device=dev).normal_(generator=g) for n in (2, 2, 4))
    cos = torch.ones((10, 32), device=dev)
    before = [x.clone() for x in (k_cache, v_cache, q)]
    for slots, positions, bit in (([64, -2, 1 << 40, -(1 << 40), 64, 65], [0] * 6, m.STATUS_BAD_SLOT),
                                  ([0, 1, 2, 3, 4, 5], [-1, 10, 11, 1 << 30, -5, 1000], m.STATUS_BAD_LENGTH)):
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        m.lora_kv_append(m.make_kv_cache(k_cache, v_cache), k, v, torch.tensor(slots, device=dev), 0, q=q,
                         position=torch.tensor(positions, dtype=torch.int32, device=dev), rope=m.Rope(cos, cos), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == bit
        for x, y in zip((k_cache, v_cache, q), before):
            assert torch.equal(x, y)


def test_append_many_rows(dev):
    """More rows than a grid dimension holds."""
    rows = 70001
    g = torch.Generator(device=dev).manual_seed(4)
    k_cache, v_cache = make_cache(dev, torch.float16, 1, rows // 16 + 1, 16, 1, 16, False, g)
    k, v = (torch.empty((rows, 16), dtype=torch.float16, device=dev).normal_(generator=g) for _ in range(2))
    slot = torch.randperm(rows, generator=g, device=dev)
    m.lora_kv_append(m.make_kv_cache(k_cache, v_cache), k, v, slot, 0)
    for c, x in ((k_cache, k), (v_cache, v)):
        assert torch.equal(c.reshape(-1, 16)[slot], x)
