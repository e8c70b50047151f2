"""Oracle of the 4-bit key/value cache (include/wq.h, "4-bit key/value cache"):
numpy, written from the header's formulas, value by value from the layout's
addresses.  Quantization in float32 as the header states it; attention, page
bounds and sums in float64."""

from __future__ import annotations

import functools

import numpy as np

PAGE = 64


def quantize(w):
    """float values [..., D] -> (codes uint8 [..., D], S float16, Z float16 [..., D / 32])."""
    w = np.asarray(w, np.float32)
    w = np.clip(np.where(np.isnan(w), np.float32(0), w), np.float32(-65504), np.float32(65504))
    g = w.reshape(*w.shape[:-1], -1, 32)
    lo, hi = g.min(-1), g.max(-1)
    z = (lo.astype(np.float16) + np.float16(0)).astype(np.float16)
    s = ((hi - lo) / np.float32(15)).astype(np.float16)
    sf = s.astype(np.float32)[..., None]
    q = np.rint((g - z.astype(np.float32)[..., None]) / np.where(sf > 0, sf, np.float32(1)))
    q = np.where(sf > 0, np.clip(q, 0, 15), 0)
    return q.reshape(w.shape).astype(np.uint8), s, z


def dequantize(q, s, z):
    """Exact values S q + Z, float64."""
    q = q.reshape(*q.shape[:-1], -1, 32).astype(np.float64)
    v = q * s.astype(np.float64)[..., None] + z.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], -1)


@functools.lru_cache(None)
def _places(D):
    """Byte and shift of every code, and byte of every S and Z, in a page of one head."""
    G = D // 32
    w = min(4, G)
    t = np.arange(PAGE)[:, None]
    d = np.arange(D)[None, :]
    g = np.arange(G)[None, :]
    tile, u, r, i = (t // 32) * 40 * D, (t % 32) // 16, (t % 16) // 4, t % 4
    e = 4 * u + i
    nib = lambda s: (s >> 1) + 4 * (s & 1)  # noqa: E731
    kg, rc, kn = d // 32, (d % 32) // 8, nib(d % 8)
    kword = ((u * (G // w) + kg // w) * 4 + rc) * 16 + t % 16
    kbyte = tile + 4 * (kword * w + kg % w) + kn // 2
    vn = nib(e) + 0 * d
    vword = ((d // 64) * 4 + r) * 16 + d % 16
    vbyte = tile + 16 * D + 4 * (vword * 4 + (d // 16) % 4) + vn // 2
    slot = 2 * ((r * G + g) * 8 + e)
    return dict(k=(kbyte, 4 * (kn % 2) + 0 * t), v=(vbyte, 4 * (vn % 2)),
                ks=tile + 32 * D + slot, kz=tile + 34 * D + 2 * ((t % 32) * G + g),
                vs=tile + 36 * D + slot, vz=tile + 38 * D + slot)


def write_token(page, t, k, v):
    """Token t of one head's page (uint8 [80 D], changed) from k, v [D]; other bits stay."""
    P = _places(k.shape[-1])
    for x, name in ((k, "k"), (v, "v")):
        q, s, z = quantize(x)
        byte, shift = P[name][0][t], P[name][1][t]
        for half, keep in ((0, 0xF0), (4, 0x0F)):
            at = byte[shift == half]                # each byte once
            page[at] = (page[at] & np.uint8(keep)) | (q[shift == half] << np.uint8(half))
        for val, at in ((s, P[name + "s"][t]), (z, P[name + "z"][t])):
            raw = val.view(np.uint8).reshape(-1, 2)
            page[at], page[at + 1] = raw[:, 0], raw[:, 1]


def read_page(page, D):
    """One head's page (uint8 [..., 80 D]) -> exact keys, values float64 [..., 64, D],
    and what bounds a logit's rounding: |S q| + |Z| of the keys."""
    P = _places(D)

    def half(at):
        raw = page[..., at].astype(np.uint16) | (page[..., at + 1].astype(np.uint16) << 8)
        return raw.view(np.float16).astype(np.float64)

    out = []
    for name in ("k", "v"):
        byte, shift = P[name]
        q = ((page[..., byte] >> shift.astype(np.uint8)) & 15).astype(np.float64)
        s = np.repeat(half(P[name + "s"]), 32, -1)
        z = np.repeat(half(P[name + "z"]), 32, -1)
        out.append(s * q + z)
        if name == "k":
            size = np.abs(s * q) + np.abs(z)
    return out[0], out[1], size


def append(data, summary, k, v, slots):
    """data uint8 [n_pages, H, 80 D] and summary float16 (or None), changed in place."""
    began = set()
    for row, slot in enumerate(slots):
        if slot < 0 or slot >= data.shape[0] * PAGE:
            continue
        p, t = divmod(int(slot), PAGE)
        for h in range(data.shape[1]):
            write_token(data[p, h], t, k[row, h], v[row, h])
        if summary is not None:
            x = np.asarray(k[row], np.float32)
            x = np.clip(np.where(np.isnan(x), 0, x), -65504, 65504).astype(np.float16)
            if t == 0:
                summary[p, :, 0], summary[p, :, 1] = x, x
                began.add(p)
            else:
                summary[p, :, 0] = np.minimum(summary[p, :, 0], x)
                summary[p, :, 1] = np.maximum(summary[p, :, 1], x)


def plan(lens, cu, table, free):
    """-> (table, new_lens, slots, runs, taken), sequence by sequence."""
    table = table.copy()
    B, width = table.shape
    T = int(cu[-1])
    slots, runs, taken = np.full(T, -1, np.int64), [], 0
    for b in range(B):
        n, pos = int(cu[b + 1] - cu[b]), int(lens[b])
        for p in range(-(-pos // PAGE), -(-(pos + n) // PAGE)):
            if p < width:
                table[b, p] = free[taken] if taken < len(free) else -1
            taken += 1
        for i in range(n):
            p, o = divmod(pos + i, PAGE)
            if i == 0 or o == 0:
                runs.append([int(cu[b]) + i, 0])
            runs[-1][1] += 1
            if p < width and table[b, p] >= 0:
                slots[cu[b] + i] = table[b, p] * PAGE + o
    most = min(T, T // PAGE + 2 * B)
    runs += [[-1, 0]] * (most - len(runs))
    new = np.asarray(lens) + np.diff(cu)
    return table, new, slots, np.array(runs).reshape(-1, 2), taken


def rows_of(lens, cu):
    """(sequence, position) of every row."""
    out = []
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        out += [(b, int(lens[b]) - n + i) for i in range(n)]
    return out


def select(summary, q, table, lens, cu, n_sel):
    """int64 [rows, H, n_sel]."""
    with np.errstate(invalid="ignore", over="ignore"):      # infinite and huge queries
        return _select(summary, q, table, lens, cu, n_sel)


def _select(summary, q, table, lens, cu, n_sel):
    n_pages, H = summary.shape[:2]
    T, heads, D = q.shape
    q = np.asarray(q, np.float64)
    sel = np.full((T, H, n_sel), -1, np.int64)
    for row, (b, pos) in enumerate(rows_of(lens, cu)):
        m = min(max(pos // PAGE + 1, 0), table.shape[1]) if pos >= 0 else 0
        for h in range(H):
            x = q[row, h * (heads // H):(h + 1) * (heads // H)]
            takes_part = np.isfinite(x).all(-1)
            score = np.full(m, -np.inf, np.float32)
            for p in range(m):
                page = table[b, p]
                if 0 <= page < n_pages:
                    s = summary[page, h].astype(np.float64)
                    s = np.maximum(x * s[0], x * s[1]).sum(-1)[takes_part]
                    score[p] = np.where(np.isnan(s), -np.inf, s).max(initial=-np.inf)
            always = np.isin(np.arange(m), (0, m - 1))
            pick = np.sort(np.lexsort((np.arange(m), -score, ~always))[:n_sel])
            sel[row, h, :len(pick)] = pick
    return sel


def attention(data, q, table, lens, cu, scale, window=0, sel=None):
    """-> out, lse, and per row and head: sum p |v| and the largest |logit| terms (float64)."""
    n_pages, H = data.shape[:2]
    T, heads, D = q.shape
    q = np.asarray(q, np.float64)
    R = heads // H
    out, lse = np.zeros((T, heads, D)), np.full((T, heads), -np.inf)
    size, top = np.zeros((T, heads, D)), np.zeros((T, heads))
    rows = rows_of(lens, cu)
    held = {}
    for row, (b, pos) in enumerate(rows):
        for h in range(H):
            m = min(max(pos // PAGE + 1, 0), table.shape[1]) if pos >= 0 else 0
            pages = range(m) if sel is None else [p for p in sel[row, h] if 0 <= p < m]
            pages = [p for p in pages if 0 <= table[b, p] < n_pages]
            if not pages:
                continue
            for p in pages:
                if (b, h, p) not in held:
                    held[b, h, p] = read_page(data[table[b, p], h], D)
            at = np.concatenate([p * PAGE + np.arange(PAGE) for p in pages])
            ok = (at <= pos) & ((at > pos - window) if window else True)
            if not ok.any():
                continue
            k, v, ks = (np.concatenate([held[b, h, p][j] for p in pages])[ok] for j in range(3))
            x = q[row, h * R:(h + 1) * R]
            z = scale * (x @ k.T)
            mx = z.max(-1, keepdims=True)
            e = np.exp(z - mx)
            l = e.sum(-1, keepdims=True)
            hs = slice(h * R, (h + 1) * R)
            out[row, hs] = (e / l) @ v
            size[row, hs] = (e / l) @ np.abs(v)
            lse[row, hs] = (mx + np.log(l))[:, 0]
            top[row, hs] = abs(scale) * (np.abs(x) @ ks.T).max(-1)
    return out, lse, size, top
