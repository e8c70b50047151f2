"""Oracle of the 8-bit key/value cache, the attention weights of its tokens, their
eviction, and the norm and rotation of queries and keys (include/wq.h): numpy, written
from the header's formulas, value by value from the layout's addresses.  Quantization in
float32 as the header states it; everything else in float64."""

from __future__ import annotations

import functools

import numpy as np

from oracle.kv4_oracle import PAGE, rows_of

BLOCK, LEAST = 16, -24


def finite(w):
    w = np.asarray(w, np.float32)
    return np.clip(np.where(np.isnan(w), np.float32(0), w), np.float32(-65504), np.float32(65504))


def exponent(most):
    """The smallest e >= -24 with most 2^-e < 127.5."""
    e = LEAST
    while not float(most) * 2.0 ** -e < 127.5:
        e += 1
    return e


def rint(x):
    return np.rint(np.asarray(x, np.float64)).astype(np.int64)


@functools.lru_cache(None)
def places(D):
    """Byte of every code of a page of one head: keys, values, [64, D]."""
    t, d = np.arange(PAGE)[:, None], np.arange(D)[None, :]
    u, l, r, i = t // 16, t % 16, t % 16 // 4, t % 4
    k = (((u * (D // 64) + d // 64) * 4 + d % 32 // 8) * 16 + l) * 16 + d // 32 % 2 * 8 + d % 8
    v = 64 * D + (((d // 16) * 4 + r) * 16 + d % 16) * 16 + u * 4 + i
    return k, v


def append_page(page, exps, o, k, v):
    """Tokens o .. o + len(k) - 1 of one head's page (uint8 [128 D], int8 [8]; changed)."""
    for w, at, first in ((finite(k), places(k.shape[-1])[0], 0), (finite(v), places(v.shape[-1])[1], 4)):
        n = len(w)
        for u in range(o // BLOCK, (o + n - 1) // BLOCK + 1):
            a, b = max(o, u * BLOCK), min(o + n, (u + 1) * BLOCK)
            e = exponent(np.abs(w[a - o:b - o]).max())
            if a > u * BLOCK:
                was = int(np.clip(int(exps[first + u]), LEAST, 10))
                e = max(e, was)
                old = at[u * BLOCK:a]
                if e > was:
                    page[old] = (rint((page[old].astype(np.float64) - 128) * 2.0 ** (was - e)) + 128).astype(np.uint8)
            exps[first + u] = e
            page[at[a:b]] = (rint(w[a - o:b - o].astype(np.float64) * 2.0 ** -e) + 128).astype(np.uint8)


def append(data, exps, k, v, slots, runs):
    """data uint8 [n_pages, H, 128 D] and exps int8 [n_pages, H, 8], changed in place."""
    for first, n in np.asarray(runs).reshape(-1, 2):
        if n <= 0 or not 0 <= slots[first] < data.shape[0] * PAGE:
            continue
        p, o = divmod(int(slots[first]), PAGE)
        for h in range(data.shape[1]):
            append_page(data[p, h], exps[p, h], o, k[first:first + n, h], v[first:first + n, h])


def read_page(page, exps, D):
    """One head's page -> exact keys, values float64 [64, D]."""
    u = np.arange(PAGE) // BLOCK
    return tuple((page[at].astype(np.float64) - 128) * 2.0 ** exps[first + u].astype(np.float64)[:, None]
                 for at, first in zip(places(D), (0, 4)))


def _seen(data, table, b, pos, window):
    """Positions that a row sees."""
    m = min(max(pos // PAGE + 1, 0), table.shape[1]) if pos >= 0 else 0
    pages = [p for p in range(m) if 0 <= table[b, p] < data.shape[0]]
    at = np.concatenate([p * PAGE + np.arange(PAGE) for p in pages] + [np.zeros(0, np.int64)]).astype(np.int64)
    return at[(at <= pos) & ((at > pos - window) if window else True)]


def attention(data, exps, q, table, lens, cu, scale, window=0):
    """-> out, lse, and per row and head: sum p |v| and the largest |logit| terms (float64)."""
    H = data.shape[1]
    T, heads, D = q.shape
    q = np.asarray(q, np.float64)
    R = heads // H
    out, lse = np.zeros((T, heads, D)), np.full((T, heads), -np.inf)
    size, top = np.zeros((T, heads, D)), np.zeros((T, heads))
    held = {}
    for row, (b, pos) in enumerate(rows_of(lens, cu)):
        at = _seen(data, table, b, pos, window)
        if not len(at):
            continue
        for h in range(H):
            if (b, h) not in held:
                held[b, h] = [read_page(data[p, h], exps[p, h], D) if 0 <= p < data.shape[0] else
                              (np.zeros((PAGE, D)),) * 2 for p in table[b]]
                held[b, h] = [np.concatenate(x) for x in zip(*held[b, h])]
            k, v = (x[at] for x in held[b, h])
            hs = slice(h * R, (h + 1) * R)
            x = q[row, hs]
            z = scale * (x @ k.T)
            mx = z.max(-1, keepdims=True)
            e = np.exp(z - mx)
            l = e.sum(-1, keepdims=True)
            out[row, hs] = (e / l) @ v
            size[row, hs] = (e / l) @ np.abs(v)
            lse[row, hs] = (mx + np.log(l))[:, 0]
            top[row, hs] = abs(scale) * (np.abs(x) @ np.abs(k).T).max(-1)
    return out, lse, size, top


def accumulate(data, exps, q, lse, table, lens, cu, held, mass, scale, window=0):
    """-> the new mass, the largest |logit| terms of a (sequence, head), and how many
    weights it sums (float64)."""
    H = data.shape[1]
    T, heads, D = q.shape
    q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
    R, S = heads // H, mass.shape[2]
    mass = np.array(mass, np.float64)
    top, count = np.zeros(mass.shape[:2] + (1,)), np.zeros(mass.shape[:2] + (1,))
    for b, n in enumerate(lens):
        n = min(int(n), S, PAGE * table.shape[1])
        mass[b, :, max(int(held[b]), 0):max(n, 0)] = 0
    for row, (b, pos) in enumerate(rows_of(lens, cu)):
        at = _seen(data, table, b, pos, window)
        for h in range(H):
            hs = slice(h * R, (h + 1) * R)
            on = np.isfinite(lse[row, hs])
            if not len(at) or not on.any():
                continue
            k = np.zeros((len(at), D))
            for p in np.unique(at // PAGE):
                k[at // PAGE == p] = read_page(data[table[b, p], h], exps[table[b, p], h], D)[0][at[at // PAGE == p] % PAGE]
            x = q[row, hs][on]
            w = np.exp(scale * (x @ k.T) - lse[row, hs][on][:, None]).sum(0)
            mass[b, h, at[at < S]] += w[at < S]
            top[b, h] = max(top[b, h, 0], abs(scale) * (np.abs(x) @ np.abs(k).T).max())
            count[b, h] += on.sum()
    return mass, top, count


def evict(data, exps, mass, table, lens, keep, recent, free, new_mass):
    """data and exps changed in place -> kept, new_table, new_lens, new_mass, taken."""
    B, H, _ = mass.shape
    width, D = table.shape[1], data.shape[2] // 128
    kept, new_table, new_mass = np.full((B, H, keep), -1, np.int64), table.copy(), new_mass.copy()
    new_lens, taken, need = np.zeros(B, np.int64), 0, -(-keep // PAGE)
    source, source_exps = data.copy(), exps.copy()
    # tokens past the masses have none
    mass = np.concatenate([mass, np.zeros((B, H, max(0, PAGE * width - mass.shape[2])), mass.dtype)], -1)
    for b in range(B):
        n = min(max(int(lens[b]), 0), PAGE * width)
        new_lens[b] = min(n, keep)
        if n > keep:
            new_table[b] = -1
            for p in range(need):
                new_table[b, p] = free[taken + p] if taken + p < len(free) else -1
            taken += need
        for h in range(H):
            pick = list(range(n))
            if n > keep:
                m = np.where(np.isnan(mass[b, h]), -np.inf, mass[b, h])
                # NaN is below every number, minus infinity too
                order = sorted(range(n - recent), key=lambda t: (np.isnan(mass[b, h, t]), -m[t], t))
                pick = sorted(order[:keep - recent]) + list(range(n - recent, n))
            kept[b, h, :len(pick)] = pick
            new_mass[b, h, :len(pick)] = mass[b, h, pick]
            if n <= keep:
                continue
            for first, at in zip((0, 4), places(D)):
                for j in range(0, keep, BLOCK):
                    page = new_table[b, j // PAGE]
                    if not 0 <= page < data.shape[0]:
                        continue
                    codes, e = [], []
                    for t in pick[j:j + BLOCK]:
                        src = table[b, t // PAGE]
                        ok = 0 <= src < data.shape[0]
                        codes.append(source[src, h][at[t % PAGE]].astype(np.float64) - 128 if ok else np.zeros(D))
                        e.append(int(np.clip(int(source_exps[src, h, first + t % PAGE // BLOCK]), LEAST, 10)) if ok else LEAST)
                    exps[page, h, first + j % PAGE // BLOCK] = max(e)
                    for x, (c, f) in enumerate(zip(codes, e)):
                        data[page, h][at[j % PAGE + x]] = (rint(c * 2.0 ** (f - max(e))) + 128).astype(np.uint8)
    return kept, new_table, new_lens, new_mass, taken


def norm_rope(x, weight, positions, inv_freq, eps, neighbours=False):
    """x [rows, heads, D] -> the result, and the absolute sum that bounds its rounding."""
    y = np.asarray(x, np.float64)
    if eps is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, np.float64)
    size = np.abs(y)
    n = 0 if inv_freq is None else len(inv_freq)
    if n:
        t = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
        j = np.arange(n)
        a, b = (2 * j, 2 * j + 1) if neighbours else (j, n + j)
        out = y.copy()
        out[..., a], out[..., b] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t), y[..., b] * np.cos(t) + y[..., a] * np.sin(t)
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
        y = out
    return y, size
