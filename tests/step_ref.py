"""Definitions in 64 bits of the norm, the 8-bit rows, the base product and the next token, with the tolerances that follow from
the types and from fp32's rounding (u = 2^-24)."""
import torch

U = 2.0 ** -24
BLOCK = 128
LEAST = 2.0 ** -126
E4M3 = torch.float8_e4m3fn
STEP = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # between a type's smallest numbers


def norm(x, residual, weight, eps):
    """(h, v) and the relative bound of v in fp32."""
    h = x.double() + (0 if residual is None else residual.double())
    v = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        v = v * weight.double()
    # h: u. The sum of squares: at most 32 additions in a thread, 10 in the tree, with 2 u of each square's h; halved
    # by the root. Division, eps, root, reciprocal, two products: 6 u.
    return h, v, (1 + (32 + 10 + 2) / 2 + 6) * U


def gated(x, gate):
    v = x.double()
    if gate is None:
        return v, torch.zeros_like(v)
    g = gate.double()
    # the documented error of __expf, 2 + 1.173 |g| ulp (of 2 u), its part in 1 + exp(-g) at most all of it; __fdividef 2 ulp; sum, two
    # products: 3 u
    return v * g * torch.sigmoid(g), (2 * (2 + 1.173 * g.abs()) + 4 + 3) * U


def within(got, want, rel, what):
    """A 16-bit output: half a step of its type beside the fp32 result's own error."""
    t = got.dtype
    g, top = got.double(), torch.finfo(t).max
    bound = want.abs() * (torch.finfo(t).eps / 2 * (1 + rel) + rel) + STEP[t]
    # (what rounds beyond the type's range is an infinity)
    fine = ((g - want).abs() <= bound) | (g == want) | (torch.isinf(g) & (want.abs() * (1 + rel) >= top) & (g.sign() == want.sign()))
    fine |= torch.isnan(g) & torch.isnan(want)
    assert bool(fine.all()), f"{what}: {int((~fine).sum())} of {fine.numel()} off, worst {float((g - want).abs().nan_to_num().max()):.3g}"


def blocks_of(v, fill=0.0):
    n = -(-v.shape[1] // BLOCK)
    return torch.nn.functional.pad(v, (0, n * BLOCK - v.shape[1]), value=fill).reshape(v.shape[0], n, BLOCK)


def check_rows8(q, scale, v, rel, what):
    """8-bit rows against the values v (64 bits, off by `rel` of themselves in fp32)."""
    rel = rel + torch.zeros_like(v)
    amax = blocks_of(v.abs()).amax(-1)
    want = torch.maximum(amax / 448, torch.full_like(amax, LEAST))
    off = blocks_of(rel).amax(-1) + 2 * U  # the product with 1/448, itself rounded
    assert bool(((scale.double() - want).abs() <= want * off).all()), f"{what}: scales off by {float(((scale.double() - want) / want).abs().max()):.3g}"
    z = blocks_of(v) / scale.double()[..., None]  # of the scale as it is
    got = blocks_of(q.float().double())
    # half a step of e4m3 (3 bits behind the point, exponents from -6) and the error of v, of the reciprocal and the product
    e = torch.floor(torch.log2(torch.maximum(z.abs(), got.abs()).clamp(min=2.0 ** -6)))
    bound = torch.exp2(e - 4) + z.abs() * (blocks_of(rel) + 3 * U)
    fine = ((got - z).abs() <= bound) | ((got.abs() == 448) & (z.abs() >= 448) & (z.abs() <= 448 * (1 + 1e-5)))
    assert bool(fine.all()), f"{what}: {int((~fine).sum())} values off"


def values8(q, scale, rows):
    s = scale.double() if rows == 1 else scale.double().repeat_interleave(rows, 0)[: q.shape[0]]
    return q.float().double() * s.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def matmul(x, x_scale, w, w_scale):
    """y and its bound in fp32: at most 128 additions in a block, whatever their order, two roundings for each block's
    scale and product, and an addition a block, each u of the sum of the products' magnitudes."""
    a, b = values8(x, x_scale, 1), values8(w, w_scale, BLOCK)
    blocks = -(-x.shape[1] // BLOCK)
    return a @ b.t(), (a.abs() @ b.abs().t()) * ((128 + 3 + blocks) * U)


def sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    """(token, logprob, margin): margin is how far the nearest decision was from a border, relative to its sum."""
    token, logprob, margin = [], [], []
    for i in range(logits.shape[0]):
        at = lambda a, d: d if a is None else a[i].item()  # noqa: E731
        x = logits[i].float().double()
        x = torch.where(torch.isnan(x), -torch.inf, x)
        t, k, p, least = at(temperature, 1.0), at(top_k, 0), at(top_p, 1.0), at(min_p, 0.0)
        x, ids = torch.sort(x, descending=True, stable=True)
        if x[0] == -torch.inf:
            token.append(-1), logprob.append(-float("inf")), margin.append(1.0)
            continue
        y = torch.where(x == x[0], 0.0, (x - x[0]) / (t if t > 0 else 1.0))
        w = torch.where(x == -torch.inf, 0.0, torch.exp(y))
        n = 1 if not t > 0 else min(k, len(x)) if k > 0 else len(x)
        cum, near = w.cumsum(0), 1.0
        if p < 1:
            goal = max(p, 0.0) * cum[n - 1]
            if n > 1 and p > 0:
                near = min(near, float(((cum[:n] - goal).abs() / cum[n - 1]).min()))
            n = min(n, max(1, int((cum < goal).sum()) + 1))
        if least > 0:
            if n > 1:
                near = min(near, float((w[:n] / least - 1).abs().min()))
            n = min(n, max(1, int((w >= least).sum())))
        u = uniform[i].item()
        u = min(u, 1 - 2.0 ** -24) if u > 0 else 0.0
        goal = u * cum[n - 1]
        j = int((cum <= goal).sum())
        if n > 1 and u > 0:
            near = min(near, float(((cum[:n] - goal).abs() / cum[n - 1]).min()))
        token.append(int(ids[j])), logprob.append(float(y[j] - torch.log(cum[n - 1]))), margin.append(near)
    return token, logprob, margin
