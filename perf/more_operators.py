"""Workloads of a serving step's operators between the adapters and the cache: the root-mean-square norm
with the residual's addition and 8-bit output, the quantiser of the other projections' inputs (with the
gate of an MLP), the base product in 8-bit floating point with a scale for each block of 128, and the
choice of the next token from given random numbers.

Each case names its operator in ``op``. ``prepare`` makes what a serving program holds before the call;
``run`` is one call, through the library where ``own`` is true and in plain torch otherwise; ``exact`` is
the definition in 64 bits. 8-bit rows are returned as e4m3 values beside their scales.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NORM, QUANT, MATMUL, SAMPLE = "norm", "quantize", "matmul", "sample"
E4M3 = torch.float8_e4m3fn
BLOCK = 128
TOP = 448.0           # the largest e4m3 value
LEAST = 2.0 ** -126   # of a scale
EPS = 1e-5


def listed():
    return [
        # a decode step of 32 requests, Llama-2-7B width: the residual's sum, x for the adapters and in 8 bits
        dict(name="norm-decode-32", op=NORM, rows=32, width=4096, dtype="bf16", residual=True, out=True, q=True),
        # a prefill batch of eight prompts, 12604 rows of Llama-2-13B width
        dict(name="norm-prefill-12604", op=NORM, rows=12604, width=5120, dtype="bf16", residual=True, out=True, q=True),
        # the last norm before the logits, an odd number of rows and a last block of 56: 16 bits only, no residual
        dict(name="norm-odd-1003", op=NORM, rows=1003, width=2744, dtype="fp16", residual=False, out=True, q=False),
        # silu(gate) * up of a decode step, Llama-2-7B MLP, for the down projection and its adapters
        dict(name="gate-decode-32", op=QUANT, rows=32, width=11008, dtype="bf16", gate=True, out=True),
        # the same of the prefill batch, Llama-2-13B MLP
        dict(name="gate-prefill-12604", op=QUANT, rows=12604, width=13824, dtype="bf16", gate=True, out=True),
        # one request's output projection, Llama-2-7B: latency counts
        dict(name="matmul-1", op=MATMUL, rows=1, d_in=4096, d_out=4096, dtype="bf16"),
        # a decode step's gate and up in one product, Llama-2-7B: the weights' bytes count
        dict(name="matmul-decode-32", op=MATMUL, rows=32, d_in=4096, d_out=22016, dtype="bf16"),
        # odd sizes: rows, a last block of k of 16 and a last block of n of 104
        dict(name="matmul-odd-213", op=MATMUL, rows=213, d_in=2064, d_out=1000, dtype="fp16"),
        # a large decode batch, Llama-2-70B MLP
        dict(name="matmul-256", op=MATMUL, rows=256, d_in=8192, d_out=28672, dtype="bf16"),
        # the prefill batch's gate, Llama-2-13B: the largest, bound by the tensor cores
        dict(name="matmul-prefill-12604", op=MATMUL, rows=12604, d_in=5120, d_out=13824, dtype="bf16"),
        # one request's next token, top-k and top-p
        dict(name="sample-1", op=SAMPLE, rows=1, vocab=32000, dtype="fp32", top_k=50, top_p=0.9, min_p=0.0, greedy=0.0),
        # a large batch over a large, odd vocabulary; the tenants' settings differ from none to all, some greedy
        dict(name="sample-256", op=SAMPLE, rows=256, vocab=128001, dtype="fp32", top_k=1000, top_p=0.7, min_p=0.1, greedy=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, dtype = rng.choice([NORM, QUANT, MATMUL, MATMUL, SAMPLE, SAMPLE]), rng.choice(["bf16", "bf16", "fp16"])
    if op == MATMUL:
        d_in, d_out = 16 * _log(rng, 8, 1024), 8 * _log(rng, 8, 3584)
        # at most the listed prefill product's work
        rows = _log(rng, 1, max(1, min(12604, 12604 * 5120 * 13824 // (d_in * d_out))))
        return dict(op=op, rows=rows, d_in=d_in, d_out=d_out, dtype=dtype)
    if op == SAMPLE:
        return dict(op=op, rows=_log(rng, 1, 256), vocab=_log(rng, 1000, 128001), dtype=rng.choice(["fp32", "fp32", dtype]),
                    top_k=rng.choice([0, _log(rng, 1, 2000)]), top_p=rng.choice([1.0, rng.uniform(0.1, 0.99)]),
                    min_p=rng.choice([0.0, rng.uniform(0.001, 0.3)]), greedy=rng.choice([0.0, 0.0, 0.3]))
    width = 8 * _log(rng, 8, 2048)
    rows = _log(rng, 1, 12604 * 5120 // max(width, 5120))
    if op == NORM:
        out = rng.random() < 0.7
        return dict(op=op, rows=rows, width=width, dtype=dtype, residual=rng.random() < 0.7, out=out,
                    q=not out or rng.random() < 0.7)
    return dict(op=op, rows=rows, width=width, dtype=dtype, gate=rng.random() < 0.6, out=rng.random() < 0.6)


def _ceil(a, b):
    return -(-a // b)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, dtype, g, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _quantized(v):
    """fp32 [rows][width] as e4m3 values and a scale for each row's block of 128."""
    rows, width = v.shape
    blocks = _ceil(width, BLOCK)
    v = torch.nn.functional.pad(v, (0, blocks * BLOCK - width)).reshape(rows, blocks, BLOCK)
    scale = (v.abs().amax(-1) / TOP).clamp(min=LEAST)
    q = (v / scale[..., None]).clamp(-TOP, TOP).to(E4M3)
    return q.reshape(rows, -1)[:, :width].contiguous(), scale


def _quantized64(v):
    """The same in 64 bits, e4m3 rounding written out: a step of 2^(e - 3) for values of 2^e and more, e from -6 on."""
    scale = torch.stack([b.abs().amax(-1) for b in v.split(BLOCK, -1)], -1) / TOP
    scale = torch.maximum(scale, torch.full_like(scale, LEAST))
    z = v / scale.repeat_interleave(BLOCK, -1)[:, : v.shape[1]]
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(z / step) * step, -TOP, TOP), scale


# ---- norm --------------------------------------------------------------------------------------


def _norm_prepare(case, g):
    n, d, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
    # a residual stream: a few channels are far larger than the others
    channel = torch.exp(_normal((d,), torch.float32, g, 0.6))
    channel[torch.randperm(d, generator=g, device="cuda")[: max(1, d // 500)]] *= 20
    s = dict(x=(_normal((n, d), torch.float32, g) * (0.3 * channel)).to(dt), weight=(1 + _normal((d,), torch.float32, g, 0.2)).to(dt))
    s["residual"] = (_normal((n, d), torch.float32, g) * channel).to(dt) if case["residual"] else None
    s["want"] = case["out"], case["q"]
    if own:
        import adapter_gemv_gb300 as m
        s["made"] = dict(residual_out=_empty((n, d), dt) if case["residual"] else None,
                         out=_empty((n, d), dt) if case["out"] else None,
                         q=_empty((n, d), E4M3) if case["q"] else None,
                         q_scale=_empty((n, _ceil(d, BLOCK)), torch.float32) if case["q"] else None)
        s["call"] = m.RmsNorm(s["x"], s["weight"], EPS, residual=s["residual"], **s["made"])
    return s


def _norm_run(s):
    if own:
        s["call"]()
        return s["made"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    v = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out, eight = s["want"]
    q, scale = _quantized(v) if eight else (None, None)
    dt = s["x"].dtype
    return dict(residual_out=h.to(dt) if s["residual"] is not None else None, out=v.to(dt) if out else None, q=q, q_scale=scale)


def _norm_exact(case, seed):
    s = _norm_prepare(case, _generator(seed))
    h = s["x"].double()
    if case["residual"]:
        h += s["residual"].double()
    mean = torch.linalg.vector_norm(h, dim=-1, keepdim=True).square() / case["width"]
    v = s["weight"].double() * (h / torch.sqrt(mean + EPS))
    q, scale = _quantized64(v) if case["q"] else (None, None)
    return dict(residual_out=h if case["residual"] else None, out=v if case["out"] else None, q=q, q_scale=scale)


def _norm_work(case):
    n, d = case["rows"], case["width"]
    each = 2 * (1 + 2 * case["residual"] + case["out"]) * d + case["q"] * (d + 4 * _ceil(d, BLOCK))
    return {"bytes": n * each + 2 * d, "flops": n * d * (4 + case["residual"] + 3 * case["q"])}


# ---- quantize ----------------------------------------------------------------------------------


def _quant_prepare(case, g):
    n, d, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
    # gate and up are the halves of one projection's output
    both = _normal((n, 2 * d if case["gate"] else d), dt, g, 1.5)
    s = dict(x=both[:, -d:], gate=both[:, :d] if case["gate"] else None, out=case["out"])
    if own:
        import adapter_gemv_gb300 as m
        s["made"] = dict(q=_empty((n, d), E4M3), q_scale=_empty((n, _ceil(d, BLOCK)), torch.float32),
                         out=_empty((n, d), dt) if case["out"] else None)
        s["call"] = m.Quantize(s["x"], gate=s["gate"], **s["made"])
    return s


def _quant_run(s):
    if own:
        s["call"]()
        return s["made"]
    v = s["x"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        v = v * (gate / (1 + torch.exp(-gate)))
    q, scale = _quantized(v)
    return dict(q=q, q_scale=scale, out=v.to(s["x"].dtype) if s["out"] else None)


def _quant_exact(case, seed):
    s = _quant_prepare(case, _generator(seed))
    v = s["x"].double()
    if case["gate"]:
        v = v * s["gate"].double() * torch.sigmoid(s["gate"].double())
    q, scale = _quantized64(v)
    return dict(q=q, q_scale=scale, out=v if case["out"] else None)


def _quant_work(case):
    n, d = case["rows"], case["width"]
    return {"bytes": n * (2 * d * (1 + case["gate"] + case["out"]) + d + 4 * _ceil(d, BLOCK)),
            "flops": n * d * (3 + 5 * case["gate"])}


# ---- matmul ------------------------------------------------------------------------------------


def _matmul_prepare(case, g):
    n, k, m_ = case["rows"], case["d_in"], case["d_out"]
    x, x_scale = _quantized(_normal((n, k), torch.float32, g) * torch.exp(_normal((k,), torch.float32, g, 0.5)))
    # weights quantised by blocks of 128 x 128, as a checkpoint holds them
    rows, cols = _ceil(m_, BLOCK), _ceil(k, BLOCK)
    w_scale = (torch.rand((rows, cols), generator=g, device="cuda") * 1.5 + 0.5) * (4 / TOP / math.sqrt(k))
    w = _normal((m_, k), torch.float32, g, TOP / 4).clamp_(-TOP, TOP).to(E4M3)
    s = dict(x=x, x_scale=x_scale, w=w, w_scale=w_scale, dtype=DTYPES[case["dtype"]])
    if own:
        import adapter_gemv_gb300 as m
        s["y"] = _empty((n, m_), s["dtype"])
        s["call"] = m.Fp8Matmul(s["y"], x, x_scale, w, w_scale)
    return s


def _scaled(q, scale, rows):
    """fp32 values of q: a scale for each block of `rows` rows and 128 columns."""
    s = scale if rows == 1 else scale.repeat_interleave(rows, 0)[: q.shape[0]]
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def _matmul_run(s):
    if own:
        s["call"]()
        return s["y"]
    return torch.matmul(_scaled(s["x"], s["x_scale"], 1), _scaled(s["w"], s["w_scale"], BLOCK).t()).to(s["dtype"])


def _matmul_exact(case, seed):
    s = _matmul_prepare(case, _generator(seed))
    y = torch.zeros((case["rows"], case["d_out"]), dtype=torch.float64, device="cuda")
    part = max(1, 32768 // case["d_out"]) * BLOCK  # some blocks of k at a time
    for k in range(0, case["d_in"], part):
        end = min(k + part, case["d_in"])
        at = torch.arange(k, end, device="cuda") // BLOCK
        a = s["x"][:, k:end].double() * s["x_scale"].double()[:, at]
        b = s["w"][:, k:end].double() * s["w_scale"].double()[:, at][torch.arange(case["d_out"], device="cuda") // BLOCK]
        y += torch.einsum("ik,nk->in", a, b)
    return y


def _matmul_work(case):
    n, k, m_ = case["rows"], case["d_in"], case["d_out"]
    blocks = _ceil(k, BLOCK)
    return {"bytes": n * (k + 4 * blocks) + m_ * k + 4 * blocks * _ceil(m_, BLOCK) + 2 * n * m_, "flops": 2 * n * k * m_}


# ---- sample ------------------------------------------------------------------------------------


def _sample_prepare(case, g):
    n, vocab, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    u = lambda lo, hi: torch.empty(n, device="cuda").uniform_(lo, hi, generator=g)  # noqa: E731
    x = _normal((n, vocab), torch.float32, g, 2.5)
    # the text's likely continuations stand out
    likely = torch.randint(vocab, (n, 200), generator=g, device="cuda")
    x.scatter_add_(1, likely, torch.empty((n, 200), device="cuda").exponential_(1 / 3.0, generator=g))
    part = lambda p: torch.rand(n, generator=g, device="cuda") < p  # noqa: E731
    s = dict(logits=x.to(dt), uniform=torch.rand(n, generator=g, device="cuda"),
             temperature=torch.where(part(case["greedy"]), 0.0, u(0.3, 1.5)))
    k, lo, least = case["top_k"], case["top_p"], case["min_p"]
    top_k = torch.randint(1, max(k, 1) + 1, (n,), generator=g, device="cuda") if n > 1 else torch.full((n,), k, device="cuda")
    # in a batch every second request goes without each of the limits
    s["top_k"] = torch.where(part(0.5 if n > 1 else 1.0), top_k, 0).to(torch.int32) if k else None
    s["top_p"] = torch.where(part(0.5), 1.0, u(lo, 1.0)) if lo < 1 and n > 1 else torch.full((n,), lo, device="cuda") if lo < 1 else None
    s["min_p"] = torch.where(part(0.5), 0.0, u(0.0, least)) if least else None
    if own:
        import adapter_gemv_gb300 as m
        s["token"], s["logprob"] = _empty((n,), torch.int32), _empty((n,), torch.float32)
        s["call"] = m.Sample(s["token"], s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                             top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
    return s


def _sample_run(s):
    if own:
        s["call"]()
        return dict(token=s["token"], logprob=s["logprob"])
    # in 64 bits throughout: which token a random number falls on is decided at borders
    x, vocab = s["logits"].float(), s["logits"].shape[1]
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    x, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    x = x.double()
    y = (x - x[:, :1]) / torch.where(greedy, 1.0, t)
    w = torch.exp(y)
    mass = w.cumsum(-1)
    k = s["top_k"].long()[:, None] if s["top_k"] is not None else torch.zeros_like(greedy, dtype=torch.int64)
    k = torch.where(greedy, 1, torch.where(k > 0, k.clamp(max=vocab), vocab))
    rank = torch.arange(vocab, device=x.device)[None]
    keep = rank < k
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        keep &= (mass - w < p * mass.gather(1, k - 1)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep[:, 0] = True
    total = mass.gather(1, keep.sum(-1, keepdim=True) - 1)
    at = (mass <= s["uniform"].double()[:, None] * total).sum(-1, keepdim=True)
    logprob = y.gather(1, at) - total.log()
    return dict(token=ids.gather(1, at)[:, 0].to(torch.int32), logprob=logprob[:, 0].float())


def _sample_exact(case, seed):
    s = _sample_prepare(case, _generator(seed))
    found = []
    for i in range(case["rows"]):
        x, t, u = s["logits"][i].double(), float(s["temperature"][i]), float(s["uniform"][i])
        p = torch.softmax(x / t, -1) if t > 0 else (x == x.max()).double()
        p = torch.sort(p, descending=True).values
        n = int(s["top_k"][i]) if s["top_k"] is not None else 0
        n = 1 if t <= 0 else n if 0 < n < case["vocab"] else case["vocab"]
        p = p[:n]
        limit = float(s["top_p"][i]) if s["top_p"] is not None else 1.0
        if limit < 1:
            before = torch.cat([torch.zeros_like(p[:1]), p.cumsum(-1)[:-1]])
            p = p[: max(1, int((before < limit * p.sum()).sum()))]
        if s["min_p"] is not None:
            p = p[: max(1, int((p >= float(s["min_p"][i]) * p[0]).sum()))]
        p = p / p.sum()
        at = int(torch.searchsorted(p.cumsum(-1), torch.tensor([u], dtype=torch.float64, device="cuda"), right=True))
        found.append(torch.log(p[min(at, p.numel() - 1)]))
    return dict(token=None, logprob=torch.stack(found))


def _sample_work(case):
    n, vocab = case["rows"], case["vocab"]
    return {"bytes": n * (vocab * (4 if case["dtype"] == "fp32" else 2) + 28), "flops": 4 * n * vocab}


# ---- the interface ------------------------------------------------------------------------------


def prepare(case, seed):
    s = {NORM: _norm_prepare, QUANT: _quant_prepare, MATMUL: _matmul_prepare, SAMPLE: _sample_prepare}[case["op"]](
        case, _generator(seed))
    s["op"] = case["op"]
    return s


def run(state):
    return {NORM: _norm_run, QUANT: _quant_run, MATMUL: _matmul_run, SAMPLE: _sample_run}[state["op"]](state)


def exact(case, seed):
    return {NORM: _norm_exact, QUANT: _quant_exact, MATMUL: _matmul_exact, SAMPLE: _sample_exact}[case["op"]](case, seed)


def work(case):
    return {NORM: _norm_work, QUANT: _quant_work, MATMUL: _matmul_work, SAMPLE: _sample_work}[case["op"]](case)
