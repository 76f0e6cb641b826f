"""Workloads of the serving operators around the adapters: a decode step's cache layout, the write
into the paged key-value cache, the attention that reads it, and the per-request logit adjustment.

Each case names its operator in ``op``. ``prepare`` makes what a serving program holds before the
call; ``run`` is one call, through the library where ``own`` is true and in plain torch otherwise;
``exact`` is the definition in 64 bits. Lengths are spread geometrically between two bounds, so that
``work`` knows them, and dealt to the requests in a seeded order.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LAYOUT, APPEND, ATTENTION, LOGITS = "layout", "append", "attention", "logits"


def listed():
    return [
        # the layout of a decode step: 32 requests, a token each (the batch of the Llama-2-7B decode workload)
        dict(name="layout-decode-32", op=LAYOUT, requests=32, prompts=0, prompt_lo=0, prompt_hi=0, released=1,
             len_lo=40, len_hi=4000, page_tokens=16, padding=0),
        # a mixed batch: 3 prompts of 300 to 2000 tokens beside 64 decode rows, rows padded to a captured graph's size
        dict(name="layout-mixed-67", op=LAYOUT, requests=67, prompts=3, prompt_lo=300, prompt_hi=2000, released=0,
             len_lo=40, len_hi=4000, page_tokens=16, padding=61),
        # the largest: 4096 requests, 64 of them prompts, some leaving
        dict(name="layout-4096", op=LAYOUT, requests=4096, prompts=64, prompt_lo=128, prompt_hi=2048, released=101,
             len_lo=16, len_hi=4096, page_tokens=16, padding=0),
        # a decode step's new rows: Llama-2-7B heads
        dict(name="append-decode-32", op=APPEND, rows=32, q_heads=32, kv_heads=32, head_dim=128, rotary_dim=128,
             interleaved=False, page_tokens=16, heads_first=False, dtype="bf16", padding=0),
        # a prefill batch of eight prompts, 12604 rows of Llama-2-13B heads
        dict(name="append-prefill-12604", op=APPEND, rows=12604, q_heads=40, kv_heads=40, head_dim=128, rotary_dim=128,
             interleaved=False, page_tokens=16, heads_first=False, dtype="bf16", padding=4),
        # one short request alone: latency counts
        dict(name="attend-1x61", op=ATTENTION, requests=1, rows_per_request=1, len_lo=61, len_hi=61, q_heads=32,
             kv_heads=32, head_dim=128, page_tokens=16, heads_first=False, dtype="bf16", window=0),
        # a decode step of 32 requests, Llama-2-7B heads (a key-value head for every query head)
        dict(name="attend-32-mha", op=ATTENTION, requests=32, rows_per_request=1, len_lo=40, len_hi=4000, q_heads=32,
             kv_heads=32, head_dim=128, page_tokens=16, heads_first=False, dtype="bf16", window=0),
        # a decode step of 256 requests, Llama-2-70B heads (8 query heads share a key-value head): the largest
        dict(name="attend-256-gqa8", op=ATTENTION, requests=256, rows_per_request=1, len_lo=200, len_hi=4096,
             q_heads=64, kv_heads=8, head_dim=128, page_tokens=32, heads_first=True, dtype="bf16", window=0),
        # one long document: the length has to be split over the whole GPU
        dict(name="attend-1x131071", op=ATTENTION, requests=1, rows_per_request=1, len_lo=131071, len_hi=131071,
             q_heads=64, kv_heads=8, head_dim=128, page_tokens=64, heads_first=False, dtype="fp16", window=0),
        # odd sizes: heads of 80, groups of 3, pages of 24, three drafted tokens a request, a sliding window
        dict(name="attend-odd", op=ATTENTION, requests=37, rows_per_request=3, len_lo=3, len_hi=2777, q_heads=15,
             kv_heads=5, head_dim=80, page_tokens=24, heads_first=False, dtype="fp16", window=1000),
        # one request's next token
        dict(name="logits-1", op=LOGITS, rows=1, vocab=32000, dtype="fp32", history=700, biases=20, masks=1, masked=1.0),
        # a large batch over a large, odd vocabulary; every second request is held to a grammar
        dict(name="logits-256", op=LOGITS, rows=256, vocab=128001, dtype="fp32", history=4096, biases=300, masks=16,
             masked=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([LAYOUT, APPEND, ATTENTION, ATTENTION, LOGITS])
    page_tokens = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    if op == LAYOUT:
        requests = _log(rng, 1, 4096)
        return dict(op=op, requests=requests, prompts=rng.randint(0, max(1, requests // 64)), prompt_lo=16,
                    prompt_hi=_log(rng, 17, 2048), released=rng.randint(0, requests // 16), len_lo=1,
                    len_hi=_log(rng, 2, 4096), page_tokens=rng.choice([8, 16, 24, 32, 64]), padding=rng.choice([0, 0, rng.randint(1, 200)]))
    if op == LOGITS:
        rows = _log(rng, 1, 256)
        return dict(op=op, rows=rows, vocab=_log(rng, 30000, 128001), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    history=_log(rng, 1, 4096), biases=rng.choice([0, rng.randint(1, 300)]), masks=rng.randint(1, 16),
                    masked=rng.choice([0.0, 0.5, 1.0]))
    kv_heads, group = rng.choice([(32, 1), (40, 1), (8, 8), (8, 4), (1, 16), (4, 7), (5, 3), (2, 12)])
    head_dim = rng.choice([64, 80, 128, 128, 256])
    common = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page_tokens=page_tokens,
                  heads_first=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))
    if op == APPEND:
        # at most the listed prefill batch's elements
        most = 12604 * 120 * 128 // ((group + 2) * kv_heads * head_dim)
        return dict(common, rows=_log(rng, 1, most), rotary_dim=rng.choice([head_dim, head_dim // 2 // 16 * 16, 0]),
                    interleaved=rng.random() < 0.3, padding=rng.choice([0, rng.randint(1, 9)]))
    rows_per_request = rng.choice([1, 1, 1, rng.randint(2, 4)])
    # at most half the listed largest batch's cache, whatever the spread of the lengths
    budget = 256 * 1280 * 8 * 128 // 2 // (kv_heads * head_dim * rows_per_request)
    requests = min(_log(rng, 1, 256), max(1, budget // 64))
    len_hi = min(_log(rng, rows_per_request, 131072), max(8, budget // requests))
    len_lo = max(rows_per_request, min(len_hi, _log(rng, 1, len_hi)))
    return dict(common, requests=requests, rows_per_request=rows_per_request, len_lo=len_lo, len_hi=max(len_lo, len_hi),
                window=rng.choice([0, 0, rng.randint(1, 4096)]))


def _spread(lo, hi, n):
    """n lengths from lo to hi, geometrically spread."""
    lo = max(1, lo)
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dealt(values, g):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t[torch.randperm(t.numel(), generator=g, device="cuda")].contiguous()


def _normal(shape, dtype, g, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _cache(pages, case, g):
    """K and V as [layer][page][token][head][d] views; heads_first lays a page out head by head."""
    t, h, d = case["page_tokens"], case["kv_heads"], case["head_dim"]
    shape = (1, pages, h, t, d) if case["heads_first"] else (1, pages, t, h, d)
    made = [_normal(shape, DTYPES[case["dtype"]], g) for _ in range(2)]
    return [m.transpose(2, 3) if case["heads_first"] else m for m in made]


# ---- layout ------------------------------------------------------------------------------------


def _layout_requests(case):
    """(kv_len, new_tokens) of the requests before they are dealt: prompts, leavers, decoding ones."""
    n, p = case["requests"], min(case["prompts"], case["requests"])
    r = min(case["released"], n - p)
    lens = _spread(case["len_lo"], case["len_hi"], n - p) if n > p else []
    prompts = _spread(case["prompt_lo"], case["prompt_hi"], p) if p else []
    step = max(1, (n - p) // r) if r else 1
    leave = {i * step for i in range(r)}
    return [(0, m) for m in prompts] + [(m, -1 if i in leave else 1) for i, m in enumerate(lens)]


def _layout_prepare(case, g):
    reqs, pt = _layout_requests(case), case["page_tokens"]
    both = torch.tensor(reqs, dtype=torch.int32, device="cuda")[torch.randperm(len(reqs), generator=g, device="cuda")]
    kv_len, new = both[:, 0].contiguous(), both[:, 1].contiguous()
    longest = max(max(a + max(b, 0) for a, b in reqs), 1)
    max_pages = _ceil(longest, pt)
    used = sum(_ceil(a, pt) for a, _ in reqs)
    need = sum(_ceil(a + max(b, 0), pt) - _ceil(a, pt) for a, b in reqs)
    num_pages = used + need + 64
    ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    old = (kv_len + pt - 1) // pt
    col = torch.arange(max_pages, device="cuda", dtype=torch.int32)[None]
    have = col < old[:, None]
    at = (torch.cumsum(have.reshape(-1).to(torch.int64), 0) - 1).clamp_(min=0).reshape(have.shape)
    table = torch.where(have, ids[at], torch.full_like(col, -1)).contiguous()
    count = num_pages - used
    head = int(torch.randint(num_pages, (1,), generator=g, device="cuda"))
    ring = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(count, device="cuda")) % num_pages] = ids[used:]
    rows = sum(max(b, 0) for _, b in reqs) + case["padding"]
    s = dict(kv_len=kv_len, new_tokens=new, page_table=table, free_ring=ring, page_tokens=pt, num_rows=rows,
             free_state=torch.tensor([head, count], dtype=torch.int32, device="cuda"),
             adapter_slot=torch.randint(-1, 64, (len(reqs),), generator=g, device="cuda", dtype=torch.int32))
    if own:
        # the step's buffers: a serving program makes them once and reuses them for every step
        import adapter_gemv_gb300 as m
        s["batch"] = m.KvBatch(s["new_tokens"], s["kv_len"], s["page_table"], s["free_ring"], s["free_state"], pt, rows,
                               adapter_slot=s["adapter_slot"], kv_len_out=torch.empty_like(kv_len),
                               free_state_out=torch.empty_like(s["free_state"]))
    return s


LAYOUT_OUT = ("page_table", "free_ring", "free_state_out", "kv_len_out", "seg_offsets", "seg_slot", "row_request",
              "position", "cache_slot", "row_slot")


def _layout_run(s):
    if own:
        import adapter_gemv_gb300 as m
        m.lora_kv_layout(s["batch"])
        return {k: getattr(s["batch"], k) for k in LAYOUT_OUT}
    pt, n, table, ring = s["page_tokens"], s["num_rows"], s["page_table"], s["free_ring"]
    new, old_len, i32 = s["new_tokens"].long(), s["kv_len"].long(), torch.int32
    pages, (head, count) = ring.numel(), s["free_state"].long().unbind()
    grow, leaves = new.clamp(min=0), new < 0
    old, want = (old_len + pt - 1) // pt, (old_len + grow + pt - 1) // pt
    need, back = want - old, torch.where(leaves, old, 0)
    ends, taken, given = grow.cumsum(0), need.cumsum(0), back.cumsum(0)
    col = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (col >= old[:, None]) & (col < want[:, None])
    popped = (head + (taken - need)[:, None] + col - old[:, None]) % pages
    table.copy_(torch.where(fresh, ring[popped], table))
    gone = leaves[:, None] & (col < old[:, None])
    to = torch.where(gone, (head + count + (given - back)[:, None] + col) % pages, pages)
    wide = torch.cat([ring, ring[:1]]).scatter(0, to.reshape(-1), table.reshape(-1))
    ring.copy_(wide[:pages])
    row = torch.arange(n, device=table.device)
    req = torch.searchsorted(ends, row, right=True)
    real = req < new.numel()
    at = req.clamp(max=new.numel() - 1)
    pos = old_len[at] + row - (ends - grow)[at]
    cell = pos.clamp(min=0, max=table.shape[1] * pt - 1)
    slot = table[at, cell // pt].long() * pt + cell % pt
    zero, last = torch.zeros_like(ends[:1]), torch.full_like(ends[:1], n)
    return dict(page_table=table, free_ring=ring,
                free_state_out=torch.stack([(head + taken[-1]) % pages, count - taken[-1] + given[-1]]).to(i32),
                kv_len_out=torch.where(leaves, 0, old_len + grow).to(i32),
                seg_offsets=torch.cat([zero, ends, last]).to(i32),
                seg_slot=torch.cat([s["adapter_slot"], torch.full_like(s["adapter_slot"][:1], -1)]),
                row_request=torch.where(real, at, -1).to(i32), position=torch.where(real, pos, -1).to(i32),
                cache_slot=torch.where(real, slot, -1),
                row_slot=torch.where(real, s["adapter_slot"][at], -1).to(i32))


def _layout_work(case):
    reqs, pt = _layout_requests(case), case["page_tokens"]
    rows = sum(max(b, 0) for _, b in reqs) + case["padding"]
    new = sum(_ceil(a + max(b, 0), pt) - _ceil(a, pt) for a, b in reqs)
    back = sum(_ceil(a, pt) for a, b in reqs if b < 0)
    return {"bytes": len(reqs) * 24 + rows * 20 + (new + back) * 8, "flops": 0}


# ---- append ------------------------------------------------------------------------------------

MAX_POSITION = 4096


def _append_prepare(case, g):
    n, hq, hk, d, pt = (case[k] for k in ("rows", "q_heads", "kv_heads", "head_dim", "page_tokens"))
    dt, total = DTYPES[case["dtype"]], case["rows"] + case["padding"]
    # q, k and v are column blocks of one projection's output
    qkv = _normal((total, (hq + 2 * hk) * d), dt, g)
    pages = _ceil(n, pt) + 3
    k, v = _cache(pages, case, g)
    slot = torch.randperm(pages * pt, generator=g, device="cuda")[:n]
    s = dict(q=qkv[:, : hq * d], k=qkv[:, hq * d: (hq + hk) * d], v=qkv[:, (hq + hk) * d:], k_cache=k, v_cache=v,
             cache_slot=torch.cat([slot, torch.full((case["padding"],), -1, device="cuda")]),
             position=torch.randint(0, MAX_POSITION, (total,), generator=g, device="cuda", dtype=torch.int32),
             q_out=torch.zeros((total, hq * d), dtype=dt, device="cuda"), rotary_dim=case["rotary_dim"],
             interleaved=case["interleaved"], heads=(hq, hk, d))
    half = case["rotary_dim"] // 2
    angle = torch.arange(MAX_POSITION, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(half, device="cuda") / max(half, 1))[None]
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        import adapter_gemv_gb300 as m
        rope = m.Rope(s["cos"], s["sin"], interleaved=case["interleaved"]) if half else None
        s["call"] = m.KvAppend(m.make_kv_cache(k, v), s["k"], s["v"], s["cache_slot"], 0, q=s["q"], q_out=s["q_out"],
                               position=s["position"], rope=rope)
    return s


def _rotated(x, s):
    """x [rows][heads][d] in fp32, rotated by its rows' positions."""
    rot, half = s["rotary_dim"], s["rotary_dim"] // 2
    if not rot:
        return x
    cos, sin = (s[n][s["position"].long()][:, None] for n in ("cos", "sin"))
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :half], x[..., half:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ra, rb], -1).flatten(-2) if s["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append_run(s):
    if own:
        s["call"]()
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    hq, hk, d = s["heads"]
    n, dt, slot = s["q"].shape[0], s["q"].dtype, s["cache_slot"]
    pt, used = s["k_cache"].shape[2], slot >= 0
    q, k = (_rotated(s[x].float().reshape(n, h, d), s).to(dt) for x, h in (("q", hq), ("k", hk)))
    at = slot.clamp(min=0)
    # rows without a slot write their first used neighbour's values again
    src = torch.where(used, torch.arange(n, device=slot.device), 0)
    at = at[src]
    s["k_cache"][0].index_put_((at // pt, at % pt), k[src])
    s["v_cache"][0].index_put_((at // pt, at % pt), s["v"].reshape(n, hk, d)[src])
    s["q_out"].copy_(torch.where(used[:, None], q.reshape(n, hq * d), s["q_out"]))
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _append_exact(case, seed):
    s = _append_prepare(case, _generator(seed))
    hq, hk, d = s["heads"]
    pt, rot, half = case["page_tokens"], case["rotary_dim"], case["rotary_dim"] // 2
    used = torch.nonzero(s["cache_slot"] >= 0).flatten()
    slot, pos = s["cache_slot"][used], s["position"][used].long()

    def turned(x, heads):
        x = x[used].double().reshape(-1, heads, d)
        if rot:
            z = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
            first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
            second = first + (1 if case["interleaved"] else half)
            r = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = r.real, r.imag
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache[0, slot // pt, slot % pt] = turned(s["k"], hk)
    v_cache[0, slot // pt, slot % pt] = s["v"][used].double().reshape(-1, hk, d)
    q = s["q_out"].double()
    q[used] = turned(s["q"], hq).reshape(-1, hq * d)
    return dict(q=q, k_cache=k_cache, v_cache=v_cache)


def _append_work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    row = 2 * 2 * (hq + 2 * hk) * d + 12
    table = min(case["rows"], MAX_POSITION) * 4 * case["rotary_dim"]
    return {"bytes": case["rows"] * row + table, "flops": case["rows"] * 3 * (hq + hk) * case["rotary_dim"]}


# ---- attention ---------------------------------------------------------------------------------


def _attention_prepare(case, g):
    n, per, hq, d, pt = (case[k] for k in ("requests", "rows_per_request", "q_heads", "head_dim", "page_tokens"))
    lens = _dealt(_spread(case["len_lo"], case["len_hi"], n), g)
    max_pages = _ceil(max(case["len_hi"], case["len_lo"]), pt)
    used = (lens + pt - 1) // pt
    pages = sum(_ceil(m, pt) for m in _spread(case["len_lo"], case["len_hi"], n)) + 5
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(max_pages, device="cuda", dtype=torch.int32)[None]
    have = col < used[:, None]
    at = (torch.cumsum(have.reshape(-1).to(torch.int64), 0) - 1).clamp_(min=0).reshape(have.shape)
    table = torch.where(have, ids[at], torch.full_like(col, -1)).contiguous()
    k, v = _cache(pages, case, g)
    # the last rows_per_request tokens of a request are its new ones, one query row each
    position = (lens[:, None] - per + torch.arange(per, device="cuda", dtype=torch.int32)[None]).reshape(-1)
    request = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(per)
    dt = DTYPES[case["dtype"]]
    s = dict(q=_normal((n * per, hq * d), dt, g), out=torch.empty((n * per, hq * d), dtype=dt, device="cuda"),
             lse=torch.empty((n * per, hq), dtype=torch.float32, device="cuda"), k_cache=k, v_cache=v, page_table=table,
             position=position.contiguous(), row_request=request, scale=d ** -0.5, window=case["window"], q_heads=hq)
    if own:
        import adapter_gemv_gb300 as m
        cache = m.make_kv_cache(k, v)
        s["call"] = m.KvAttention(s["out"], s["q"], cache, table, s["position"], 0, m.kv_attention_workspace(cache, hq),
                                  row_request=request, lse=s["lse"], scale=s["scale"], window=s["window"])
    return s


def _attention_run(s):
    if own:
        s["call"]()
        return dict(out=s["out"], lse=s["lse"])
    (rows, _), hq = s["q"].shape, s["q_heads"]
    _, _, pt, hk, d = s["k_cache"].shape
    table = s["page_table"][s["row_request"].long()].long()
    t = torch.arange(table.shape[1] * pt, device=table.device)[None]
    pos = s["position"].long()[:, None]
    seen = (t <= pos) & (t > pos - s["window"]) if s["window"] else t <= pos
    table = table.clamp(min=0)
    q = s["q"].float().reshape(rows, hk, hq // hk, d)
    k = s["k_cache"][0][table].reshape(rows, -1, hk, d).permute(0, 2, 3, 1).float()
    score = torch.matmul(q, k) * s["scale"]
    del k
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    v = s["v_cache"][0][table].reshape(rows, -1, hk, d).permute(0, 2, 1, 3).float()
    out = torch.matmul(weight, v) / total
    return dict(out=out.reshape(rows, -1).to(s["q"].dtype), lse=(top + total.log()).reshape(rows, hq))


def _attention_exact(case, seed):
    s = _attention_prepare(case, _generator(seed))
    _, _, pt, hk, d = s["k_cache"].shape
    hq, out, lse = s["q_heads"], [], []
    for i, (r, p) in enumerate(zip(s["row_request"].tolist(), s["position"].tolist())):
        first = max(0, p + 1 - s["window"]) if s["window"] else 0
        t = torch.arange(first, p + 1, device="cuda")
        page = s["page_table"][r, t // pt].long()
        k, v = (s[n][0, page, t % pt].double() for n in ("k_cache", "v_cache"))
        q = s["q"][i].double().reshape(hk, hq // hk, d)
        score = torch.einsum("hgd,thd->hgt", q, k) * s["scale"]
        lse.append(torch.logsumexp(score, -1).reshape(-1))
        out.append(torch.einsum("hgt,thd->hgd", torch.softmax(score, -1), v).reshape(-1))
    return dict(out=torch.stack(out), lse=torch.stack(lse))


def _attention_work(case):
    n, per, hq, hk, d = (case[k] for k in ("requests", "rows_per_request", "q_heads", "kv_heads", "head_dim"))
    lens, w = _spread(case["len_lo"], case["len_hi"], n), case["window"]
    # a request's rows read one cache, from the first row's first token to the last row's last
    read = sum(min(m, w + per - 1) if w else m for m in lens)
    seen = sum(min(m - per + 1 + j, w) if w else m - per + 1 + j for m in lens for j in range(per))
    return {"bytes": read * hk * d * 4 + n * per * hq * (d * 4 + 4), "flops": 4 * seen * hq * d}


# ---- logits ------------------------------------------------------------------------------------


def _logits_prepare(case, g):
    n, vocab, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    u = lambda lo, hi: torch.empty(n, device="cuda").uniform_(lo, hi, generator=g)  # noqa: E731
    total = _dealt(_spread(max(1, case["history"] // 8), case["history"], n), g)
    # tokens of a text: few are frequent (a power law over the vocabulary)
    x = torch.rand((n, case["history"]), generator=g, device="cuda")
    tokens = (vocab ** x - 1).long().clamp(max=vocab - 1)
    tokens = (tokens * 7919 % vocab).to(torch.int32)
    b = case["biases"]
    bias_token = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:b] for _ in range(n)]).to(torch.int32)
    words = _ceil(vocab, 32)
    grammar = torch.randint(-(1 << 31), 1 << 31, (case["masks"], words), generator=g, device="cuda").to(torch.int32)
    held = torch.rand(n, generator=g, device="cuda") < case["masked"]
    pick = torch.randint(case["masks"], (n,), generator=g, device="cuda", dtype=torch.int32)
    s = dict(logits=_normal((n, vocab), dt, g, 3.0), out=torch.empty((n, vocab), dtype=dt, device="cuda"),
             tokens=tokens, total_len=total, prompt_len=(total * u(0.0, 1.0)).to(torch.int32), repetition=u(1.0, 1.3),
             presence=u(-0.5, 1.0), frequency=u(-0.1, 0.5), temperature=u(0.3, 1.5),
             bias_offsets=torch.arange(n + 1, device="cuda", dtype=torch.int32) * b,
             bias_token=bias_token.reshape(-1), bias_value=_normal((n * b,), torch.float32, g, 2.0), mask=grammar,
             mask_index=torch.where(held, pick, -1).to(torch.int32))
    if own:
        import adapter_gemv_gb300 as m
        s["call"] = m.LogitsAdjust(s["out"], s["logits"], tokens=s["tokens"], prompt_len=s["prompt_len"],
                                   total_len=s["total_len"], repetition=s["repetition"], presence=s["presence"],
                                   frequency=s["frequency"], temperature=s["temperature"],
                                   bias=(s["bias_offsets"], s["bias_token"], s["bias_value"]), mask=s["mask"],
                                   mask_index=s["mask_index"])
    return s


def _logits_run(s):
    if own:
        s["call"]()
        return s["out"]
    n, vocab = s["logits"].shape
    at = torch.arange(s["tokens"].shape[1], device="cuda")[None]
    known, made = at < s["total_len"][:, None], at >= s["prompt_len"][:, None]
    ids = s["tokens"].long()
    ever = torch.zeros((n, vocab), device="cuda").scatter_add_(1, ids, known.float())
    count = torch.zeros((n, vocab), device="cuda").scatter_add_(1, ids, (known & made).float())
    rep, pres, freq, temp = (s[k][:, None] for k in ("repetition", "presence", "frequency", "temperature"))
    x = s["logits"].float()
    x = torch.where(ever > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * count - pres * (count > 0)
    b = s["bias_token"].numel() // n
    if b:
        x = x.scatter_add(1, s["bias_token"].long().reshape(n, b), s["bias_value"].reshape(n, b))
    x = x / temp
    v = torch.arange(vocab, device="cuda")
    bits = (s["mask"][s["mask_index"].long().clamp(min=0)][:, v // 32] >> (v % 32).to(torch.int32)) & 1
    barred = (bits == 0) & (s["mask_index"] >= 0)[:, None]
    return x.masked_fill(barred, float("-inf")).to(s["logits"].dtype)


def _logits_exact(case, seed):
    s = _logits_prepare(case, _generator(seed))
    n, vocab = s["logits"].shape
    out = s["logits"].double()
    for i in range(n):
        text = s["tokens"][i, : int(s["total_len"][i])].long()
        made = torch.bincount(text[int(s["prompt_len"][i]):], minlength=vocab).double()
        seen = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        seen[text] = True
        rep = s["repetition"][i].double()
        x = out[i]
        x = torch.where(seen, torch.maximum(x, x * 0) / rep + torch.minimum(x, x * 0) * rep, x)
        x = x - made * s["frequency"][i].double() - (made > 0) * s["presence"][i].double()
        lo, hi = s["bias_offsets"][i: i + 2].tolist()
        x[s["bias_token"][lo:hi].long()] += s["bias_value"][lo:hi].double()
        x = x / s["temperature"][i].double()
        j = int(s["mask_index"][i])
        if j >= 0:
            bits = s["mask"][j].long()[:, None] >> torch.arange(32, device="cuda")[None] & 1
            x[bits.reshape(-1)[:vocab] == 0] = -math.inf
        out[i] = x
    return out


def _logits_work(case):
    n, vocab = case["rows"], case["vocab"]
    size = 4 if case["dtype"] == "fp32" else 2
    held = round(case["masked"] * n)
    history = sum(_spread(max(1, case["history"] // 8), case["history"], n))
    masks = min(held, case["masks"])
    return {"bytes": n * vocab * 2 * size + 4 * history + 8 * n * case["biases"] + masks * _ceil(vocab, 32) * 4 + 32 * n,
            "flops": 6 * n * vocab}


# ---- the interface ------------------------------------------------------------------------------


def prepare(case, seed):
    s = {LAYOUT: _layout_prepare, APPEND: _append_prepare, ATTENTION: _attention_prepare,
         LOGITS: _logits_prepare}[case["op"]](case, _generator(seed))
    s["op"] = case["op"]
    return s


def run(state):
    return {LAYOUT: _layout_run, APPEND: _append_run, ATTENTION: _attention_run, LOGITS: _logits_run}[state["op"]](state)


def exact(case, seed):
    if case["op"] == LAYOUT:
        return None  # whole numbers only
    return {APPEND: _append_exact, ATTENTION: _attention_exact, LOGITS: _logits_exact}[case["op"]](case, seed)


def work(case):
    return {LAYOUT: _layout_work, APPEND: _append_work, ATTENTION: _attention_work, LOGITS: _logits_work}[case["op"]](case)
