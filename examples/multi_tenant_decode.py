"""A small decoder that serves many tenants' requests, each on its own LoRA adapter: every step of the
library together, as a serving loop runs them.

    python examples/multi_tenant_decode.py

Per step, from the requests' lengths alone (all on the GPU; the host only says how many rows there are):
  lora_kv_layout     pages and cache slots of the step's rows, and their adapter segments
  per layer          q, k, v = base products + lora_sgmv_grouped over those segments
                     lora_kv_append     rotary positions, k and v into the paged cache
                     lora_kv_attention  every row over its request's pages
                     o, gate/up, down   base products + adapters
  lora_logits_adjust the request's own penalties, biases, temperature and grammar on its logits
  lora_sample        its next token, from a random number, within its top-k, top-p and min-p
With base8 the base weights are held in 8 bits, with a scale for each block of 128 x 128:
  lora_rms_norm      the residual's sum and its norm, in 16 bits for the adapters and in 8 for the base products
  lora_quantize      the same of the attention's output, and of silu(gate) up
  lora_fp8_matmul    the base products
The weights are random: the text means nothing, but two tenants with one prompt get different texts.
"""
from __future__ import annotations

import dataclasses
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import adapter_gemv_gb300 as m
import workloads as W


@dataclasses.dataclass
class Config:
    layers: int = 2
    hidden: int = 512
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    mlp: int = 1024
    vocab: int = 2003
    adapters: int = 4
    rank: int = 16
    page_tokens: int = 16
    pages: int = 256
    max_len: int = 512
    dtype: torch.dtype = torch.bfloat16
    base8: bool = False


def blocks8(w):
    """w [d_in][d_out] as e4m3 values [d_out][d_in] and a power of two for each block of 128 x 128."""
    t = w.t().contiguous().float()
    grid = [-(-n // m.FP8_BLOCK) for n in t.shape]
    scale = torch.ones(grid, device=w.device)
    for i in range(grid[0]):
        for j in range(grid[1]):
            at = slice(i * 128, i * 128 + 128), slice(j * 128, j * 128 + 128)
            scale[i, j] = torch.exp2(torch.ceil(torch.log2(t[at].abs().amax() / 448)))
    spread = scale.repeat_interleave(128, 0)[:t.shape[0]].repeat_interleave(128, 1)[:, :t.shape[1]]
    return (t / spread).to(torch.float8_e4m3fn), scale


def values8(q, scale):
    """The [d_in][d_out] matrix that they stand for."""
    spread = scale.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return (q.float() * spread).t().contiguous()


class Model:
    """Base weights, one adapter pool per projection, rotary tables."""

    def __init__(self, c: Config, dev, seed: int = 0):
        g = W.generator(seed, dev)
        self.c, kv, qd = c, c.kv_heads * c.head_dim, c.q_heads * c.head_dim
        self.shapes = {"q": (c.hidden, qd), "k": (c.hidden, kv), "v": (c.hidden, kv), "o": (qd, c.hidden),
                       "gate": (c.hidden, c.mlp), "up": (c.hidden, c.mlp), "down": (c.mlp, c.hidden)}
        self.w = [{n: W.normal((i, o), 1.0 / i, c.dtype, g, dev) for n, (i, o) in self.shapes.items()}
                  for _ in range(c.layers)]
        if c.base8:  # (w: the values that the 8-bit weights stand for)
            self.w8 = [{n: blocks8(w) for n, w in layer.items()} for layer in self.w]
            self.w = [{n: values8(*w).to(c.dtype) for n, w in layer.items()} for layer in self.w8]
        self.pools = {n: W.stacked_pool(num_slots=c.adapters, num_layers=c.layers, r_max=c.rank, d_in=i, d_out=o,
                                        dtype=c.dtype, gen=g, device=dev) for n, (i, o) in self.shapes.items()}
        self.handles = {n: m.make_pool(p) for n, p in self.pools.items()}
        self.embed = W.normal((c.vocab, c.hidden), 1.0, c.dtype, g, dev)
        self.head = W.normal((c.hidden, c.vocab), 4.0 / c.hidden, c.dtype, g, dev)
        half = c.head_dim // 2
        angle = torch.arange(c.max_len, device=dev)[:, None] * 10000.0 ** (-torch.arange(half, device=dev) / half)[None]
        self.rope = m.Rope(angle.cos().float().contiguous(), angle.sin().float().contiguous())


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Server:
    """The requests' state on the GPU, and the steps. A request's place (0 .. places - 1) is its row in every
    per-request array; places without a request have length 0."""

    def __init__(self, model: Model, places: int, dev):
        c, i32 = model.c, dict(dtype=torch.int32, device=dev)
        self.model, self.places, self.dev = model, places, dev
        shape = (c.layers, c.pages, c.page_tokens, c.kv_heads, c.head_dim)
        self.cache = m.make_kv_cache(*(torch.zeros(shape, dtype=c.dtype, device=dev) for _ in range(2)))
        self.workspace = m.kv_attention_workspace(self.cache, c.q_heads)
        self.kv_len = torch.zeros(places, **i32)
        self.adapter_slot = torch.full((places,), -1, **i32)
        self.page_table = torch.full((places, c.max_len // c.page_tokens), -1, **i32)
        self.free_ring, self.free_state = torch.arange(c.pages, **i32), torch.tensor([0, c.pages], **i32)
        # each request's text and sampling parameters
        self.tokens = torch.zeros((places, c.max_len), **i32)
        self.prompt_len, self.total_len = torch.zeros(places, **i32), torch.zeros(places, **i32)
        f32 = dict(dtype=torch.float32, device=dev)
        self.repetition, self.temperature = torch.ones(places, **f32), torch.ones(places, **f32)
        self.presence, self.frequency = torch.zeros(places, **f32), torch.zeros(places, **f32)
        self.top_k, self.top_p, self.min_p = torch.zeros(places, **i32), torch.ones(places, **f32), torch.zeros(places, **f32)
        self.mask = torch.full((1, (c.vocab + 31) // 32), -1, **i32)  # grammar 0; -1 (none) until a request has one
        self.mask_index = torch.full((places,), -1, **i32)
        self.status = torch.zeros(1, **i32)

    def start(self, place: int, prompt, adapter: int, **sampling) -> None:
        self.tokens[place, :len(prompt)] = torch.tensor(prompt, dtype=torch.int32)
        self.prompt_len[place] = self.total_len[place] = len(prompt)
        self.adapter_slot[place] = adapter
        for name in ("repetition", "temperature", "presence", "frequency", "mask_index", "top_k", "top_p", "min_p"):
            getattr(self, name)[place] = sampling.get(name, {"repetition": 1, "temperature": 1, "mask_index": -1, "top_p": 1}.get(name, 0))

    def step(self, new: list, uniform=None) -> torch.Tensor:
        """new[place]: tokens to run of the request's text beyond what the cache holds (a new request: its prompt;
        else 1), 0: none, -1: the request leaves. Returns the adjusted logits [places][vocab]; the next token of
        every request that ran, the likeliest or that of its random number in uniform [places], is appended to its text."""
        c, rows = self.model.c, sum(max(n, 0) for n in new)
        before = self.kv_len.clone()
        batch = m.KvBatch(torch.tensor(new, dtype=torch.int32, device=self.dev), self.kv_len, self.page_table, self.free_ring,
                          self.free_state, c.page_tokens, rows, adapter_slot=self.adapter_slot)
        m.lora_kv_layout(batch, self.status)
        left = (before > 0) & (self.kv_len == 0)
        self.total_len.masked_fill_(left, 0), self.prompt_len.masked_fill_(left, 0)
        if rows == 0:
            return torch.empty((self.places, 0), device=self.dev)
        at = batch.position.long()
        x = self.model.embed[self.tokens[batch.row_request.long(), at].long()]
        if c.base8:
            x = self._layers8(x, batch, max(new))
        else:
            for layer in range(c.layers):
                x = self._layer(layer, x, batch, max(new))
            x = norm(x)
        last = (batch.seg_offsets[1:self.places + 1] - 1).clamp(min=0).long()
        logits = torch.matmul(x[last], self.model.head).float()
        ran = torch.tensor([i if n > 0 else -1 for i, n in enumerate(new)], dtype=torch.int32, device=self.dev)
        m.lora_logits_adjust(logits, logits, row_request=ran, tokens=self.tokens, prompt_len=self.prompt_len,
                             total_len=self.total_len, repetition=self.repetition, presence=self.presence,
                             frequency=self.frequency, temperature=self.temperature, mask=self.mask,
                             mask_index=self.mask_index, status=self.status)
        # the cache holds the whole text: its next token follows
        grown = (ran >= 0) & (self.kv_len == self.total_len)
        where = self.total_len.clamp(max=c.max_len - 1).long()[:, None]
        if uniform is None:
            picked = logits.argmax(-1).to(torch.int32)
        else:  # (the temperature is in the logits)
            picked = torch.zeros_like(self.total_len)
            m.lora_sample(picked, logits, uniform, row_request=ran, top_k=self.top_k, top_p=self.top_p, min_p=self.min_p,
                          status=self.status)
        nxt = torch.where(grown, picked, self.tokens.gather(1, where)[:, 0])
        self.tokens.scatter_(1, where, nxt[:, None])
        self.total_len += grown
        return logits

    def _project(self, names, x, layer, batch):
        """x W + the adapters' delta, for projections that read the same x."""
        ys = [torch.matmul(x, self.model.w[layer][n]) for n in names]
        v = [torch.empty((x.shape[0], self.model.c.rank), dtype=torch.float32, device=self.dev) for _ in names]
        m.lora_sgmv_grouped([(y, x, self.model.handles[n], layer, s) for n, y, s in zip(names, ys, v)], batch.seg_offsets,
                            batch.seg_slot, self.status)
        return ys

    def _layer(self, layer, x, batch, rows_per_request):
        q, k, v = self._project(("q", "k", "v"), norm(x), layer, batch)
        m.lora_kv_append(self.cache, k, v, batch.cache_slot, layer, q=q, position=batch.position, rope=self.model.rope,
                         status=self.status)
        out = torch.empty_like(q)
        m.lora_kv_attention_ex(out, q, self.cache, self.page_table, batch.position, layer, self.workspace, rows_per_request,
                               row_request=batch.row_request, status=self.status)
        x = x + self._project(("o",), out, layer, batch)[0]
        gate, up = self._project(("gate", "up"), norm(x), layer, batch)
        return x + self._project(("down",), torch.nn.functional.silu(gate) * up, layer, batch)[0]


    def _rows8(self, x):
        """Room for rows of x in 8 bits."""
        return (torch.empty_like(x, dtype=torch.float8_e4m3fn),
                torch.empty((x.shape[0], -(-x.shape[1] // m.FP8_BLOCK)), dtype=torch.float32, device=self.dev))

    def _project8(self, names, x, rows8, layer, batch):
        """Base products of the 8-bit rows + the adapters' delta of x."""
        c = self.model.c
        ys = [torch.empty((x.shape[0], self.model.shapes[n][1]), dtype=c.dtype, device=self.dev) for n in names]
        for n, y in zip(names, ys):
            m.lora_fp8_matmul(y, *rows8, *self.model.w8[layer][n], status=self.status)
        v = [torch.empty((x.shape[0], c.rank), dtype=torch.float32, device=self.dev) for _ in names]
        m.lora_sgmv_grouped([(y, x, self.model.handles[n], layer, s) for n, y, s in zip(names, ys, v)], batch.seg_offsets,
                            batch.seg_slot, self.status)
        return ys

    def _layers8(self, x, batch, rows_per_request):
        """All layers over the residual stream x; the norm behind them."""
        h, rows8 = torch.empty_like(x), self._rows8(x)
        m.lora_rms_norm(x, out=h, q=rows8[0], q_scale=rows8[1])
        for layer in range(self.model.c.layers):
            q, k, v = self._project8(("q", "k", "v"), h, rows8, layer, batch)
            m.lora_kv_append(self.cache, k, v, batch.cache_slot, layer, q=q, position=batch.position, rope=self.model.rope,
                             status=self.status)
            out, out8 = torch.empty_like(q), self._rows8(q)
            m.lora_kv_attention_ex(out, q, self.cache, self.page_table, batch.position, layer, self.workspace, rows_per_request,
                                   row_request=batch.row_request, status=self.status)
            m.lora_quantize(out, *out8)
            o, = self._project8(("o",), out, out8, layer, batch)
            m.lora_rms_norm(o, residual=x, out=h, q=rows8[0], q_scale=rows8[1])  # x: the sum
            gate, up = self._project8(("gate", "up"), h, rows8, layer, batch)
            act, act8 = torch.empty_like(up), self._rows8(up)
            m.lora_quantize(up, *act8, gate=gate, out=act)
            down, = self._project8(("down",), act, act8, layer, batch)
            m.lora_rms_norm(down, residual=x, out=h, q=rows8[0], q_scale=rows8[1])
        return h


def main():
    dev = torch.device("cuda:0")
    server = Server(Model(Config(base8=True), dev), places=4, dev=dev)
    numbers = torch.Generator(device=dev).manual_seed(1)
    prompt = [5, 17, 3, 99, 3, 250, 8]
    for place in range(4):  # one prompt, four tenants
        server.start(place, prompt, adapter=place, repetition=1.2, frequency=0.3, temperature=0.8, top_k=40, top_p=0.9)
    server.step([len(prompt)] * 4, torch.rand(4, generator=numbers, device=dev))
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(24):
        server.step([1] * 4, torch.rand(4, generator=numbers, device=dev))
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / 24 * 1e3
    for place in range(4):
        n = int(server.total_len[place])
        print(f"adapter {place}:", *server.tokens[place, len(prompt):n].tolist())
    server.step([-1] * 4)
    print(f"{ms:.2f} ms a step, status {int(server.status)}, free pages {server.free_state[1].item()} of {server.model.c.pages}")


if __name__ == "__main__":
    main()
