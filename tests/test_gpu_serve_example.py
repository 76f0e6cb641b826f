"""The serving loop of examples/multi_tenant_decode.py against a plain model: every request alone, its whole text
at once, in fp32, with its adapter merged into the weights."""
import importlib.util
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import adapter_gemv_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from adapter_gemv_gb300 import build
        build.build()
    spec = importlib.util.spec_from_file_location("multi_tenant_decode", os.path.join(ROOT, "examples", "multi_tenant_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod
    spec.loader.exec_module(mod)
    return mod


def plain_logits(model, text, adapter):
    """fp32 logits behind the text's last token, without cache, pages, segments or the library."""
    c = model.c
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)  # noqa: E731

    def w(layer, n):
        base = model.w[layer][n].float()
        p = model.pools[n]
        r = int(p.rank[adapter])
        return base + float(p.scale[adapter]) * p.a_t[adapter, layer, :r].float().T @ p.b[adapter, layer, :r].float()

    x = model.embed[torch.tensor(text, device=model.embed.device)].float()
    n, half = len(text), c.head_dim // 2
    cos, sin = model.rope.cos[:n, None], model.rope.sin[:n, None]

    def turn(z):
        a, b = z[..., :half], z[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    for layer in range(c.layers):
        h = norm(x)
        q = turn((h @ w(layer, "q")).reshape(n, c.q_heads, -1))
        k = turn((h @ w(layer, "k")).reshape(n, c.kv_heads, -1)).repeat_interleave(c.q_heads // c.kv_heads, 1)
        v = (h @ w(layer, "v")).reshape(n, c.kv_heads, -1).repeat_interleave(c.q_heads // c.kv_heads, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(c.head_dim)
        s = s.masked_fill(torch.ones(n, n, device=s.device).triu(1).bool(), -math.inf)
        o = torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(n, -1)
        x = x + o @ w(layer, "o")
        h = norm(x)
        x = x + (torch.nn.functional.silu(h @ w(layer, "gate")) * (h @ w(layer, "up"))) @ w(layer, "down")
    return norm(x)[-1] @ model.head.float()


def test_serving_loop_matches_the_plain_model(ex):
    """Requests that start, decode, pause and leave at different times; pages are reused. The loop's bf16 activations
    are rounded some 20 times along two layers, each to 2^-9 relative, so logits of standard deviation 2 may be
    off by a few hundredths; 0.15 of that deviation bounds the rms, and the texts follow from the logits."""
    dev = torch.device("cuda:0")
    c = ex.Config(pages=40)
    model = ex.Model(c, dev)
    server = ex.Server(model, 5, dev)
    g = torch.Generator().manual_seed(3)
    prompt = lambda n: torch.randint(0, c.vocab, (n,), generator=g).tolist()  # noqa: E731
    allowed = {5, 77, 901, 1500}
    words = torch.zeros(server.mask.shape[1], dtype=torch.int64)
    for t in allowed:
        words[t // 32] |= 1 << (t % 32)
    server.mask[0] = words.to(torch.int32).to(dev)

    live, adapters, checked = {}, {}, 0
    plan = [  # (places that start: prompt length, adapter, sampling), places that pause, places that leave
        ({0: (37, 1, {}), 3: (1, 2, dict(repetition=1.3, frequency=0.2))}, (), ()),
        ({1: (90, 0, dict(mask_index=0))}, (), ()), ({}, (3,), ()), ({4: (16, 3, dict(temperature=0.5))}, (), ()),
        ({}, (), (0,)), ({0: (200, 2, dict(presence=0.7))}, (), ()), ({}, (1, 4), ()), ({}, (), (1, 3)),
        ({1: (33, 3, {}), 3: (64, 1, {})}, (), ()), ({}, (), ()), ({}, (), ())]
    for starts, pauses, leaves in plan:
        new = [0] * 5
        for place in live:
            new[place] = -1 if place in leaves else 0 if place in pauses else 1
        for place, (n, adapter, sampling) in starts.items():
            server.start(place, prompt(n), adapter, **sampling)
            live[place], adapters[place], new[place] = sampling, adapter, n
        total = server.total_len.tolist()
        texts = {p: server.tokens[p, :total[p]].tolist() for p in range(5)}
        logits = server.step(new)
        assert int(server.status) == 0
        for place in leaves:
            del live[place]
        for place, n in enumerate(new):
            if n <= 0:
                continue
            assert int(server.kv_len[place]) == total[place] and int(server.total_len[place]) == total[place] + 1
            sampling, text = live[place], texts[place]
            got = logits[place]
            want = plain_logits(model, text, adapters[place]).double()
            made = text[int(server.prompt_len[place]):]
            rep, freq, pres = sampling.get("repetition", 1), sampling.get("frequency", 0), sampling.get("presence", 0)
            for t in set(text):
                want[t] = (want[t] / rep if want[t] > 0 else want[t] * rep) - freq * made.count(t) - pres * (t in made)
            want = want / sampling.get("temperature", 1)
            if sampling.get("mask_index", -1) >= 0:
                assert set(torch.nonzero(torch.isfinite(got)).flatten().tolist()) == allowed
                want, got = want[sorted(allowed)], got[sorted(allowed)]
            err = (got.double() - want).square().mean().sqrt()
            assert err < 0.15 * 2 / sampling.get("temperature", 1), (place, float(err))
            assert int(server.tokens[place, total[place]]) == int(logits[place].argmax())
            checked += 1
    assert checked >= 25
    new = [-1 if p in live else 0 for p in range(5)]
    server.step(new)
    assert server.free_state[1].item() == c.pages and (server.kv_len == 0).all()
    assert sorted(server.free_ring.tolist()) == list(range(c.pages))


def test_example_runs(ex, capsys):
    ex.main()
    out = capsys.readouterr().out
    assert "status 0" in out and out.count("adapter") == 4
    texts = [ln.split(":")[1] for ln in out.splitlines() if ln.startswith("adapter")]
    assert len(set(texts)) == 4  # four tenants, four texts
