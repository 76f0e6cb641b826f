"""Plain 64-bit implementations of the serving operators, request by request, for the tests: written from
the definitions in include/mlora.h, without any of the library's code."""
from __future__ import annotations

import math

import torch

# unit roundoff of the output types: half the spacing of the numbers at 1
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the smallest spacing (subnormals)
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def ceil(a, b):
    return -(-a // b)


def layout(new_tokens, kv_len, page_table, ring, state, page_tokens, num_rows, adapter_slot):
    """Lists in, dict of lists out; 'status' as the header's bits (32 NO_PAGES, 64 BAD_LENGTH, 8 BAD_PAGE)."""
    pages, (head, count) = len(ring), state
    table, ring, n = [list(r) for r in page_table], list(ring), len(kv_len)
    most = (len(table[0]) if table else 0) * page_tokens
    adapter = adapter_slot or [-1] * n
    status = 0
    if any(a < 0 or b < -1 or a + max(b, 0) > most for a, b in zip(kv_len, new_tokens)):
        status |= 64
    if sum(max(b, 0) for b in new_tokens) > num_rows and not status:
        status |= 64
    if not (0 <= head < pages and 0 <= count <= pages):
        status |= 64
    if not status:
        need = sum(ceil(a + b, page_tokens) - ceil(a, page_tokens) for a, b in zip(kv_len, new_tokens) if b >= 0)
        back = sum(ceil(a, page_tokens) for a, b in zip(kv_len, new_tokens) if b < 0)
        if need > count:
            status |= 32
        elif count + back > pages:
            status |= 64
    out = dict(row_request=[], position=[], cache_slot=[], row_slot=[], seg_offsets=[0], seg_slot=adapter + [-1],
               kv_len_out=list(kv_len), free_state_out=[head, count])
    if not status:
        taken = given = 0
        free = [ring[(head + i) % pages] for i in range(count)]
        for r, (a, b) in enumerate(zip(kv_len, new_tokens)):
            if b < 0:
                for j in range(ceil(a, page_tokens)):
                    ring[(head + count + given) % pages] = table[r][j]
                    given += 1
                out["kv_len_out"][r] = 0
            else:
                for j in range(ceil(a, page_tokens), ceil(a + b, page_tokens)):
                    table[r][j] = free[taken]
                    taken += 1
                for t in range(a, a + b):
                    page = table[r][t // page_tokens]
                    good = 0 <= page < pages
                    status |= 0 if good else 8
                    out["row_request"].append(r)
                    out["position"].append(t)
                    out["cache_slot"].append(page * page_tokens + t % page_tokens if good else -1)
                    out["row_slot"].append(adapter[r])
                out["kv_len_out"][r] = a + b
            out["seg_offsets"].append(len(out["position"]))
        out["free_state_out"] = [(head + taken) % pages, count - taken + given]
    else:
        out["seg_offsets"] += [0] * n
    for k in ("row_request", "position", "cache_slot", "row_slot"):
        out[k] += [-1] * (num_rows - len(out[k]))
    out["seg_offsets"].append(num_rows)
    return dict(out, page_table=table, free_ring=ring, status=status)


def rotate(x, pos, cos, sin, interleaved):
    """x [heads][d] (fp64), rotated at position pos; also the magnitude its fp32 rounding errors scale with."""
    y, mag = x.clone(), x.abs()
    half = cos.shape[1]
    for m in range(half):
        i, j = (2 * m, 2 * m + 1) if interleaved else (m, m + half)
        c, s = cos[pos, m].double(), sin[pos, m].double()
        y[:, i], y[:, j] = x[:, i] * c - x[:, j] * s, x[:, j] * c + x[:, i] * s
        mag[:, i] = (x[:, i] * c).abs() + (x[:, j] * s).abs()
        mag[:, j] = (x[:, j] * c).abs() + (x[:, i] * s).abs()
    return y, mag


def rotate_tol(y, mag, dtype):
    # three fp32 roundings of terms of at most mag, then one rounding to the type
    return UNIT[dtype] * y.abs() * (1 + 2.0 ** -10) + 2.0 ** -22 * mag + TINY[dtype]


def attention(q, k_cache, v_cache, layer, page_table, request, position, scale, window):
    """q [rows][hq][d] -> out, lse (fp64), and their tolerances.

    With A the largest scale * sum_d |q_d K_d| of a row's tokens and n their number, in fp32 with
    accumulation in steps of 16 (the tensor core's, which may truncate: 2^-22 a step): a score is off by at most
    ds = (d/16 + 16) 2^-22 A, a weight relatively by 2 ds + 2^-20 (exponential) + 2^-15 (kept as a pair of
    16-bit numbers), and the sums over tokens by another (n/16 + 64) 2^-22; the output is rounded once."""
    rows, hq, d = q.shape
    _, num_pages, pt, hk, _ = k_cache.shape
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(rows):
        r, p = int(request[i]), int(position[i])
        t = torch.arange(max(0, p + 1 - window) if window else 0, p + 1, device=q.device)
        if not t.numel():
            continue
        page = page_table[r, t // pt].long()
        good = (page >= 0) & (page < num_pages)
        t, page = t[good], page[good]
        if not t.numel():
            continue
        k, v = (c[layer, page, t % pt].double().repeat_interleave(hq // hk, 1) for c in (k_cache, v_cache))
        qi = q[i].double()
        s = torch.einsum("hd,thd->ht", qi, k) * scale
        a = (torch.einsum("hd,thd->ht", qi.abs(), k.abs()) * abs(scale)).amax(1)
        w = torch.softmax(s, 1)
        out[i], lse[i] = torch.einsum("ht,thd->hd", w, v), torch.logsumexp(s, 1)
        ds, steps = (d / 16 + 16) * 2.0 ** -22 * a, (t.numel() / 16 + 64) * 2.0 ** -22
        rel = 2 * ds + 2.0 ** -20 + 2.0 ** -15 + steps
        tol[i] = UNIT[q.dtype] * out[i].abs() + rel[:, None] * torch.einsum("ht,thd->hd", w, v.abs()) + TINY[q.dtype]
        ltol[i] = ds + 2.0 ** -20 + steps + 2.0 ** -22 * lse[i].abs()
    return out, lse, tol, ltol


def logits(x, request, tokens, prompt_len, total_len, repetition, presence, frequency, temperature, bias, mask,
           mask_index):
    """x [rows][vocab] -> adjusted (fp64) and the tolerance: eight fp32 roundings of the terms' magnitudes, one
    rounding to the type. Python lists and CPU tensors; None for what has no part."""
    rows, vocab = x.shape
    y = x.double().clone()
    tol = torch.zeros_like(y)
    for i in range(rows):
        r = i if request is None else int(request[i])
        if r < 0:
            continue
        seen, made = torch.zeros(vocab, dtype=torch.bool), torch.zeros(vocab, dtype=torch.float64)
        if total_len is not None:
            for j in range(int(total_len[r])):
                t = int(tokens[r, j])
                if 0 <= t < vocab:
                    seen[t] = True
                    made[t] += j >= int(prompt_len[r])
        par = [1.0 if a is None and k == 0 else 0.0 if a is None else float(a[r])
               for k, a in enumerate((repetition, presence, frequency, temperature))]
        rep, pres, freq, temp = par
        z = torch.where(seen, torch.where(y[i] > 0, y[i] / rep, y[i] * rep), y[i])
        mag = z.abs() + (freq * made).abs() + abs(pres) * (made > 0)
        z = z - freq * made - pres * (made > 0)
        if bias is not None:
            off, tok, val = bias
            add = {int(tok[e]): float(val[e]) for e in range(int(off[r]), int(off[r + 1]))}
            for t, b in add.items():
                if 0 <= t < vocab:
                    z[t] += b
                    mag[t] += abs(b)
        if temp > 0:
            z, mag = z / temp, mag / temp
        tol[i] = UNIT[x.dtype] * z.abs() + 8 * 2.0 ** -24 * mag + TINY[x.dtype]
        if mask is not None and int(mask_index[r]) >= 0:
            word = mask[int(mask_index[r])]
            for t in range(vocab):
                if not (int(word[t // 32]) >> (t % 32)) & 1:
                    z[t] = -math.inf
        y[i] = z
    return y, tol


def assert_within(got, want, tol, what):
    got, want = got.double().cpu(), want.double().cpu()
    tol = tol.double().cpu()
    assert got.shape == want.shape, what
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        at = [tuple(x) for x in torch.nonzero(bad)[:4].tolist()]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; " + "; ".join(
            f"{a}: got {got[a].item():.9g}, want {want[a].item():.9g} +- {tol[a].item():.3g}" for a in at))
