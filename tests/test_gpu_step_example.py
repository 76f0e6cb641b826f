"""The norm, the 8-bit rows and products, the adapters, the cache and the sampling as they run together: the serving loop of
examples/multi_tenant_decode.py with 8-bit base weights against a plain fp32 model, and a chain of calls in one graph."""
import pytest
import torch

import adapter_gemv_gb300 as m
import step_ref as ref
import workloads as W
from test_gpu_serve_example import ex, plain_logits  # noqa: F401

pytestmark = pytest.mark.gpu


def test_serving_loop_in_8_bits_matches_the_plain_model(ex):  # noqa: F811
    """The weights' 8-bit values are those of the plain model (powers of two as scales). What differs is the rounding of the
    products' inputs: e4m3 is off by at most 2^-4, in the mean 2.6 % of a value, independently from element to element, so each of the
    2 x 4 stages' products is off by 2.6 %, together sqrt(8) x 2.6 = 7.4 % of the logits' deviation of 2. Three times that
    bounds the rms, with the 16-bit roundings within it."""
    dev = torch.device("cuda:0")
    c = ex.Config(pages=60, base8=True)
    model = ex.Model(c, dev)
    server = ex.Server(model, 4, dev)
    g = torch.Generator().manual_seed(5)
    prompt = lambda n: torch.randint(0, c.vocab, (n,), generator=g).tolist()  # noqa: E731
    settings = [dict(top_k=30, top_p=0.8, temperature=0.7), dict(min_p=0.1, repetition=1.2), dict(top_p=0.95, temperature=1.3), {}]
    lengths = [140, 1, 37, 64]
    for place in range(4):
        server.start(place, prompt(lengths[place]), place, **settings[place])
    for new in (lengths, [1] * 4, [1, 0, 1, 1], [1] * 4, [0, 1, 0, 1]):
        total = server.total_len.tolist()
        texts = {p: server.tokens[p, :total[p]].tolist() for p in range(4)}
        u = torch.rand(4, generator=g)
        logits = server.step(list(new), u.to(dev))
        assert int(server.status) == 0
        for place in range(4):
            if not new[place]:
                continue
            s = settings[place]
            if not s.get("repetition"):
                want = plain_logits(model, texts[place], place).double() / s.get("temperature", 1)
                err = (logits[place].double() - want).square().mean().sqrt()
                assert err < 3 * 0.074 * 2 / s.get("temperature", 1), (place, float(err))
            t, _, margin = ref.sample(logits[place:place + 1].cpu(), u[place:place + 1],
                                      **{k: torch.tensor([s[k]]) for k in ("top_k", "top_p", "min_p") if k in s})
            assert margin[0] > 2.0 ** -30 and int(server.tokens[place, total[place]]) == t[0]


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_a_chain_in_one_graph(rows):
    """norm -> 8-bit product + adapters -> gate -> 8-bit product, captured once and replayed on new inputs: the bits of the
    calls one by one, on another stream; two such graphs at a time do not disturb each other."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    bf16, d, mlp, rank = torch.bfloat16, 640, 1152, 8
    g = W.generator(7, dev)
    weights = [(torch.randn(o, i, generator=g, device=dev) * 60).clamp(-448, 448).to(ref.E4M3) for i, o in ((d, 2 * mlp), (mlp, d))]
    scales = [torch.rand(-(-w.shape[0] // 128), -(-w.shape[1] // 128), generator=g, device=dev) * 1e-3 for w in weights]
    pool = m.make_pool(W.stacked_pool(num_slots=3, num_layers=1, r_max=rank, d_in=d, d_out=2 * mlp, dtype=bf16, gen=g, device=dev))
    slot = torch.arange(rows, dtype=torch.int32, device=dev) % 4 - 1

    def chain():
        e = lambda n, t=bf16: torch.empty((rows, n), dtype=t, device=dev)  # noqa: E731
        rows8 = lambda n: (e(n, ref.E4M3), e(-(-n // 128), torch.float32))  # noqa: E731
        t = dict(x=torch.zeros((rows, d), dtype=bf16, device=dev), res=torch.zeros((rows, d), dtype=bf16, device=dev), sums=e(d), h=e(d),
                 y=e(2 * mlp), act=e(mlp), z=e(d), v=e(rank, torch.float32), st=torch.zeros(1, dtype=torch.int32, device=dev))
        h8, a8 = rows8(d), rows8(mlp)
        calls = [m.RmsNorm(t["x"], residual=t["res"], residual_out=t["sums"], out=t["h"], q=h8[0], q_scale=h8[1]),
                 m.Fp8Matmul(t["y"], *h8, weights[0], scales[0], t["st"]),
                 lambda: m.lora_bgmv(t["y"], t["h"], pool, slot, 0, t["v"], t["st"]),
                 m.Quantize(t["y"][:, mlp:], *a8, gate=t["y"][:, :mlp], out=t["act"]),
                 m.Fp8Matmul(t["z"], *a8, weights[1], scales[1], t["st"])]
        return t, lambda: [c() for c in calls]

    (a, run_a), (b, run_b), (want, run) = chain(), chain(), chain()
    run_a(), run_b()
    torch.cuda.synchronize()
    graphs, streams = [torch.cuda.CUDAGraph() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for graph, r in zip(graphs, (run_a, run_b)):
        with torch.cuda.graph(graph):
            r()
    for k in range(3):
        for t in (a, b):
            t["x"].normal_(generator=g), t["res"].normal_(generator=g)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for t in (a, b):
            want["x"].copy_(t["x"]), want["res"].copy_(t["res"])
            run()
            torch.cuda.synchronize()
            assert int(t["st"]) == 0
            for name in ("sums", "h", "y", "act", "z"):
                assert torch.equal(t[name], want[name]), (k, name)
    # and the chain's own mathematics, from the rounded values between the calls
    h, v, rel = ref.norm(want["x"], want["res"], None, 1e-5)
    ref.within(want["h"], v, rel, "h")
    assert torch.isfinite(want["z"].float()).all() and (want["z"].float().abs().amax(-1) > 0).all()
