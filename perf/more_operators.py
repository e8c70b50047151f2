"""Cases and plain forms of the operators around the paged 8-bit key/value cache.

A page holds 64 tokens of every key/value head, in four blocks of 16.  A block's
keys of one head share an exponent, and so do its values: a value stands for
q 2^e, q in -127..127, where e is the smallest number from -24 on with
max |w| 2^-e < 127.5 over the block, and q = rint(w 2^-e) (float32, ties to even;
NaN counts as 0, values are clamped to +-65504).  A block that gets more tokens
keeps its exponent or raises it: the codes it has become rint(q 2^(e - e')).

A head's page is 128 D bytes of q + 128 (D = 64, 128 or 256 channels), keys then
values.  With token t = 16 u + l = 16 u + 4 r + i (l < 16, r < 4, i < 4):
    key byte    [u][d / 64][d % 32 / 8][l][d / 32 % 2][d % 8]
    value byte  [d / 16][r][d % 16][u][i]
Exponents are int8 [page][head][8]: those of the four blocks' keys, then values.

The operators:
* rotate      norm of every head of queries and keys and the rotation by position;
* append      quantizes new keys and values into their pages;
* attend      attention of the new rows over the cache (grouped heads, causal);
* accumulate  adds every cached token's softmax weights over rows and heads of a
              group to its mass, float32 [sequence][key/value head][token];
* evict       keeps the last tokens and those of most mass, in fresh pages.
"""

import math
import random

import torch

own = False

PAGE, BLOCK = 64, 16
LEAST = -24


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the new token of one chat (Llama-3-8B-shaped heads): all latency
        dict(name="rotate_1", op="rotate", rows=1, heads=32, kv=8, dim=128, rotated=128, pairs="halves", base=500000.0, type="f16"),
        # a batch of prompts
        dict(name="rotate_8190", op="rotate", rows=8190, heads=32, kv=8, dim=128, rotated=128, pairs="halves", base=10000.0,
             type="bf16"),
        # the new tokens of a large serving batch
        dict(name="append_256x1", op="append", seqs=256, new=1, longest=2047, ragged=True, kv=8, dim=128, type="bf16"),
        # a prompt's tokens, ending inside a page
        dict(name="append_3x8190", op="append", seqs=3, new=8190, longest=9000, ragged=True, kv=8, dim=128, type="f16"),
        # a short chat answered alone: one token a step
        dict(name="attend_1x500", op="attend", seqs=1, new=1, longest=500, ragged=False, heads=32, kv=8, dim=128, type="f16", window=0),
        # a serving batch, lengths spread, one idle row as a captured batch has (Llama-3-70B-shaped heads)
        dict(name="attend_32x8191", op="attend", seqs=32, new=1, longest=8191, ragged=True, heads=64, kv=8, dim=128, type="bf16",
             window=0),
        # few long documents: the cache's bytes are all that counts
        dict(name="attend_4x131072", op="attend", seqs=4, new=1, longest=131072, ragged=False, heads=32, kv=8, dim=128, type="f16",
             window=0),
        # a piece of a prompt over what is cached of it
        dict(name="attend_2x512_over_6000", op="attend", seqs=2, new=512, longest=6000, ragged=True, heads=32, kv=8, dim=128,
             type="f16", window=0),
        # what that piece looked at
        dict(name="accumulate_2x512_over_6000", op="accumulate", seqs=2, new=512, longest=6000, ragged=True, heads=32, kv=8, dim=128,
             type="f16", window=0),
        # what a step of the serving batch looked at
        dict(name="accumulate_32x8191", op="accumulate", seqs=32, new=1, longest=8191, ragged=True, heads=64, kv=8, dim=128,
             type="bf16", window=0),
        # one chat that has outgrown its budget
        dict(name="evict_1x4500", op="evict", seqs=1, longest=4500, ragged=False, kv=8, dim=128, keep=2048, recent=256),
        # a serving batch, some of it still within its budget
        dict(name="evict_16x16000", op="evict", seqs=16, longest=16000, ragged=True, kv=8, dim=128, keep=6000, recent=1000),
    ]


def _log(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "accumulate", "evict"])
    kv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, kv=kv, dim=rng.choice([64, 128, 128, 256]), ragged=rng.random() < 0.7)
    if op != "evict":
        c["type"] = rng.choice(["f16", "bf16"])
    if op in ("rotate", "attend", "accumulate"):
        c["heads"] = kv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    if op == "rotate":
        del c["ragged"]
        c["rows"] = _log(rng, 1, max(1, 330000 * 128 // ((c["heads"] + kv) * c["dim"])))
        c["rotated"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 48])
        c["pairs"], c["base"] = rng.choice(["halves", "halves", "neighbours"]), rng.choice([10000.0, 500000.0])
    elif op == "append":
        c["seqs"] = _log(rng, 1, 300)
        c["new"] = _log(rng, 1, max(1, 24000 // c["seqs"]))
        c["longest"] = c["new"] + _log(rng, 1, max(1, 60000 // c["seqs"]))
    elif op == "evict":
        c["seqs"] = _log(rng, 1, 40)
        c["longest"] = _log(rng, 100, 200000 // (c["seqs"] * max(1, c["dim"] // 128)))
        c["keep"] = max(1, int(c["longest"] * rng.uniform(0.1, 0.9)))
        c["recent"] = rng.randint(0, c["keep"])
    elif rng.random() < 0.35:
        c["seqs"], c["new"], c["window"] = rng.randint(1, 3), _log(rng, 2, 400), 0
        c["longest"] = c["new"] + _log(rng, 1, 4000)
    else:
        c["seqs"], c["new"] = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        c["longest"] = _log(rng, 5, 300000 // (c["seqs"] * max(1, c["dim"] // 128)))
        c["window"] = rng.choice([0, 0, 0, 1000])
    return c


def _lengths(case):
    """(length after the new tokens, new tokens) of every sequence."""
    n, new, longest = case["seqs"], case.get("new", 0), case["longest"]
    if not case["ragged"]:
        return [longest] * n, [new] * n
    r = random.Random(n * 1000003 + longest)
    rows = [new if new < 8 else r.randint(new // 2, new) for _ in range(n)]
    lens = [max(rows[b], r.randint(max(1, longest // 4), longest)) for b in range(n)]
    lens[r.randrange(n)] = longest
    if n > 8 and case["op"] in ("attend", "accumulate"):
        lens[r.randrange(n)] = 0  # an idle row of the batch
    return lens, rows


def _pages(tokens):
    return -(-tokens // PAGE)


def work(case):
    D, kv = case["dim"], case["kv"]
    if case["op"] == "rotate":
        n = case["rows"] * (case["heads"] + kv)
        return {"bytes": 4 * n * D + 4 * case["rows"] + 4 * D + 4 * case["rotated"], "flops": n * (4 * D + 3 * case["rotated"])}
    lens, rows = _lengths(case)
    total = sum(rows)
    if case["op"] == "append":
        return {"bytes": total * kv * D * 6 + 12 * total, "flops": 6 * total * kv * D}
    if case["op"] == "evict":
        scored = sum(lens)
        moved = sum(case["keep"] for a in lens if a > case["keep"])
        kept = sum(min(a, case["keep"]) for a in lens)
        return {"bytes": 4 * kv * scored + 8 * kv * kept + 4 * kv * D * moved, "flops": kv * scored + 4 * kv * D * moved}
    heads, w = case["heads"], case["window"]
    seen = sum(min(a, w + b - 1) if w else a for a, b in zip(lens, rows))
    pairs = sum(min(a - b + i + 1, w) if w else a - b + i + 1 for a, b in zip(lens, rows) if a for i in range(b))
    if case["op"] == "accumulate":
        return {"bytes": 2 * total * heads * D + 4 * total * heads + seen * kv * D + 8 * sum(lens) * kv, "flops": 2 * D * heads * pairs}
    return {"bytes": 4 * total * heads * D + 2 * seen * kv * D, "flops": 4 * D * heads * pairs}


# ------------------------------------------------------------- the format


def _exponent(most):
    """Exponents of blocks whose largest magnitudes are `most` (float32)."""
    m, x = torch.frexp(most)
    e = x - 7 + (m >= 127.5 / 128).int()
    return torch.where(most > 0, e, torch.full_like(e, LEAST)).clamp(min=LEAST)


def _by_token(data, D):
    """Codes int [pages, heads, 64, D] of keys and of values, from their bytes."""
    n, h, _ = data.shape
    k = data[..., :64 * D].reshape(n, h, 4, D // 64, 4, 16, 2, 8).permute(0, 1, 2, 5, 3, 6, 4, 7).reshape(n, h, PAGE, D)
    v = data[..., 64 * D:].reshape(n, h, D // 16, 4, 16, 4, 4).permute(0, 1, 5, 3, 6, 2, 4).reshape(n, h, PAGE, D)
    return k.int() - 128, v.int() - 128


def _by_byte(k, v):
    """Bytes [pages, heads, 128 D] of codes [pages, heads, 64, D]."""
    n, h, _, D = k.shape
    k = k.view(n, h, 4, 16, D // 64, 2, 4, 8).permute(0, 1, 2, 4, 6, 3, 5, 7).reshape(n, h, -1)
    v = v.view(n, h, 4, 4, 4, D // 16, 16).permute(0, 1, 5, 3, 6, 2, 4).reshape(n, h, -1)
    return (torch.cat([k, v], -1) + 128).to(torch.uint8)


def _finite(w):
    return torch.nan_to_num(w, nan=0.0).clamp(-65504.0, 65504.0)


def _scales(e, dtype):
    """2^e for each token, [..., 64, 1], from exponents [..., 4]."""
    return torch.ldexp(torch.ones((), dtype=dtype, device=e.device), e.int()).repeat_interleave(BLOCK, -1).unsqueeze(-1)


def _values(data, exps, D, dtype):
    """Keys and values [..., 64, D] of pages [..., 128 D] and their exponents."""
    lead = data.shape[:-1]
    k, v = _by_token(data.reshape(-1, 1, 128 * D), D)
    return (k.view(*lead, PAGE, D).to(dtype) * _scales(exps[..., :4], dtype),
            v.view(*lead, PAGE, D).to(dtype) * _scales(exps[..., 4:], dtype))


def _quantized(w):
    """Codes and exponents [..., 4] of whole pages of values [..., 64, D]."""
    w = _finite(w)
    e = _exponent(w.abs().unflatten(-2, (4, BLOCK)).amax((-1, -2)))
    return torch.round(w / _scales(e, torch.float32)).int(), e


# ----------------------------------------------------------------- inputs


def _dtype(case):
    return torch.float16 if case["type"] == "f16" else torch.bfloat16


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _sums(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _filled(case, n_pages, g, dev):
    """Pages of keys and values and their exponents: every channel with its own offset, some of them large."""
    h, D = case["kv"], case["dim"]
    shift = torch.randn(h, 1, D, generator=g, device=dev) * (1 + 4 * (torch.rand(h, 1, D, generator=g, device=dev) < 0.05))
    data = torch.empty(n_pages, h, 128 * D, dtype=torch.uint8, device=dev)
    exps = torch.empty(n_pages, h, 8, dtype=torch.int8, device=dev)
    for a in range(0, n_pages, 1024):
        n = min(1024, n_pages - a)
        mood = torch.randn(n, h, 1, D, generator=g, device=dev) * 0.5  # neighbours are alike
        k, ke = _quantized((torch.randn(n, h, PAGE, D, generator=g, device=dev) + mood + shift).half().float())
        v, ve = _quantized((0.6 * torch.randn(n, h, PAGE, D, generator=g, device=dev)).half().float())
        data[a:a + n], exps[a:a + n] = _by_byte(k, v), torch.cat([ke, ve], -1)
    return data, exps


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    h, D = case["kv"], case["dim"]
    if case["op"] == "rotate":
        T, H, n, t = case["rows"], case["heads"], case["rotated"], _dtype(case)
        # the projection's output: queries, keys and values of a row side by side
        x = torch.randn(T, H + 2 * h, D, generator=g, device=dev) * torch.exp(torch.randn(T, H + 2 * h, 1, generator=g, device=dev))
        x = x.to(t)
        weight = (1 + 0.2 * torch.randn(2, D, generator=g, device=dev)).to(t)
        # positions of chunks of several sequences, some of them far along
        start = torch.randint(0, 131072, (T // 1000 + 1,), generator=g, device=dev)
        at = torch.arange(T, device=dev)
        return dict(case=case, q=x[:, :H], k=x[:, H:H + h], q_weight=weight[0], k_weight=weight[1], eps=1e-6,
                    positions=(start[at // 1000] + at % 1000).int(),
                    freqs=case["base"] ** (-torch.arange(0, n, 2, dtype=torch.float64, device=dev) / n),
                    q_out=torch.empty(T, H, D, dtype=t, device=dev), k_out=torch.empty(T, h, D, dtype=t, device=dev))
    lens, rows = _lengths(case)
    B, T = len(lens), sum(rows)
    width = max(1, max(_pages(a) for a in lens))
    used = sum(_pages(a) for a in lens)
    fresh = sum(_pages(case["keep"]) for a in lens if a > case["keep"]) if case["op"] == "evict" else 0
    order = torch.randperm(used + fresh + 8, generator=g, device=dev).int()
    s = dict(case=case, cu=_ints(_sums(rows), dev), lens=_ints(lens, dev), max_new=max(rows), max_len=max(lens))
    first = _ints(_sums([_pages(a) for a in lens]), dev)
    p = torch.arange(width, device=dev, dtype=torch.int32)
    at = (first[:-1, None] + p).clamp(max=used + fresh + 7).long()
    table = torch.where(p < -(-s["lens"][:, None] // PAGE), order[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    data, exps = _filled(case, used + fresh + 8, g, dev)
    s.update(table=table, data=data, exps=exps)
    if case["op"] == "evict":
        # few tokens have most of the weight, some exactly none
        mass = torch.rand(B, h, width * PAGE, generator=g, device=dev) ** 12 * 40
        mass = mass * (torch.rand(B, h, width * PAGE, generator=g, device=dev) > 0.2)
        keep = case["keep"]
        s.update(mass=mass, free=order[used:].contiguous(), kept=torch.empty(B, h, keep, dtype=torch.int32, device=dev),
                 new_table=torch.empty_like(table), new_lens=torch.empty_like(s["lens"]), taken=torch.empty(1, dtype=torch.int32, device=dev),
                 new_mass=torch.zeros(B, h, keep, device=dev))
        return s
    t = _dtype(case)
    if case["op"] == "append":
        # keys and values are the two halves of one projection's output; some tokens are larger than those before
        kv = torch.randn(T, 2, h, D, generator=g, device=dev) * torch.exp(0.3 * torch.randn(T, 1, h, 1, generator=g, device=dev))
        kv[:, 0] += torch.randn(h, D, generator=g, device=dev) * 2
        kv = kv.to(t)
        start = [a - b for a, b in zip(lens, rows)]
        runs, at = [], 0
        for a, n in zip(start, rows):
            done = 0
            while done < n:
                m = min(n - done, PAGE - (a + done) % PAGE)
                runs.append([at + done, m])
                done += m
            at += n
        which = torch.repeat_interleave(torch.arange(B, device=dev), _ints(rows, dev).long(), output_size=T)
        pos = torch.arange(T, device=dev) - s["cu"][which] + (_ints(start, dev))[which]
        slots = table[which, pos // PAGE] * PAGE + pos % PAGE
        s.update(k=kv[:, 0], v=kv[:, 1], slots=slots.int().contiguous(), runs=_ints(runs, dev))
        return s
    q = torch.randn(T, case["heads"], D, generator=g, device=dev) * 1.5
    s.update(q=q.to(t), scale=1 / math.sqrt(D))
    if case["op"] == "attend":
        s.update(out=torch.empty(T, case["heads"], D, dtype=t, device=dev))
        return s
    # what attention over the cache gave, and the mass that the tokens before these have
    mass = torch.rand(B, h, width * PAGE, generator=g, device=dev) ** 6 * 4
    held = [a - b if a else 0 for a, b in zip(lens, rows)]
    x, seen, b, i = _logits(s)
    lse = torch.logsumexp(x.masked_fill(~seen, -math.inf), -1).view(B, h, s["max_new"], -1).transpose(1, 2).reshape(B, s["max_new"], -1)
    s.update(lse=lse[b, i].contiguous(), mass=mass, held=_ints(held, dev))
    return s


# ------------------------------------------------------------ plain forms


def _rotate(s):
    c = s["case"]
    n = c["rotated"]
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    for x, w, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        if c["pairs"] == "halves":
            a, b = y[..., :n // 2], y[..., n // 2:n]
            y[..., :n // 2], y[..., n // 2:n] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., 0:n:2], y[..., 1:n:2]
            y[..., 0:n:2], y[..., 1:n:2] = a * cos - b * sin, b * cos + a * sin
        out.copy_(y)
    return {"q": s["q_out"], "k": s["k_out"]}


def _append(s):
    data, exps, slots = s["data"], s["exps"], s["slots"].long()
    D = data.shape[-1] // 128
    first, count = s["runs"].long().unbind(1)
    page, o = slots[first] // PAGE, slots[first] % PAGE
    t = torch.arange(PAGE, device=data.device)
    new = (t >= o[:, None]) & (t < (o + count)[:, None])  # [runs, 64]
    row = (first[:, None] + t - o[:, None]).clamp(0, len(slots) - 1)
    block = new.view(-1, 4, BLOCK)
    touched = block.any(-1)[:, None]
    older = touched & ~block[:, :, 0][:, None]  # [runs, 1, 4]: the block has tokens from before
    before = (older & (t[::BLOCK] <= o[:, None, None])).repeat_interleave(BLOCK, -1) & (t < o[:, None, None])
    codes, was = _by_token(data[page], D), exps[page].int()
    out = []
    for w, q, e in ((s["k"], codes[0], was[..., :4]), (s["v"], codes[1], was[..., 4:])):
        w = torch.where(new[:, None, :, None], _finite(w[row].float()).transpose(1, 2), torch.zeros((), device=data.device))
        most = _exponent(w.abs().unflatten(-2, (4, BLOCK)).amax((-1, -2)))
        to = torch.where(older, most.maximum(e), torch.where(touched, most, e))
        fresh = torch.round(w / _scales(to, torch.float32)).int()
        moved = torch.round(q * _scales(e - to, torch.float32)).int()
        out.append((torch.where(new[:, None, :, None], fresh, torch.where(before[..., None], moved, q)), to))
    data[page] = _by_byte(out[0][0], out[1][0])
    exps[page] = torch.cat([out[0][1], out[1][1]], -1).to(torch.int8)
    return {"data": data, "exponents": exps}


def _logits(s):
    """Logits [B h, rows heads, tokens] of every sequence's rows, which of them count, and where the rows stand."""
    q, table = s["q"].float(), s["table"].long()
    T, H, D = q.shape
    B, P = table.shape
    h, n, window = s["data"].shape[1], s["max_new"], s["case"]["window"]
    b, i, pos = _by_sequence(s)
    k = _values(s["data"][table.clamp(min=0)], s["exps"][table.clamp(min=0)], D, torch.float32)[0]
    k = k.transpose(1, 2).reshape(B * h, P * PAGE, D)
    rows = torch.zeros(B, n, H, D, device=q.device)
    rows[b, i] = q * s["scale"]
    rows = rows.view(B, n, h, H // h, D).transpose(1, 2).reshape(B * h, -1, D)
    last = torch.full((B, n), -1, device=q.device)
    last[b, i] = pos
    last = last[:, None, :, None].expand(B, h, n, H // h).reshape(B * h, -1, 1)
    at = torch.arange(P * PAGE, device=q.device)
    seen = (at <= last) & (at > last - window) if window else at <= last
    return torch.matmul(rows, k.transpose(1, 2)), seen, b, i


def _by_sequence(s):
    """(sequence, number in it, position) of every row."""
    cu = s["cu"].long()
    row = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    i = row - cu[b]
    return b, i, s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _softmax(x, seen):
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _attend(s):
    table, (T, H, D) = s["table"].long(), s["q"].shape
    (B, P), h, n = table.shape, s["data"].shape[1], s["max_new"]
    x, seen, b, i = _logits(s)
    v = _values(s["data"][table.clamp(min=0)], s["exps"][table.clamp(min=0)], D, torch.float32)[1]
    o = torch.matmul(_softmax(x, seen), v.transpose(1, 2).reshape(B * h, P * PAGE, D))
    o = o.view(B, h, n, H // h, D).transpose(1, 2).reshape(B, n, H, D)
    return s["out"].copy_(o[b, i])


def _accumulate(s):
    B, h, n = len(s["lens"]), s["data"].shape[1], s["max_new"]
    x, seen, b, i = _logits(s)
    lse = torch.full((B, n, s["q"].shape[1]), math.inf, device=x.device)
    lse[b, i] = torch.where(s["lse"].isfinite(), s["lse"], torch.full_like(s["lse"], math.inf))
    lse = lse.view(B, n, h, -1).transpose(1, 2).reshape(B * h, -1, 1)
    p = torch.where(seen, torch.exp(x - lse), torch.zeros_like(x)).sum(1).view(B, h, -1)
    at = torch.arange(p.shape[-1], device=x.device)
    before = torch.where(at < s["held"][:, None, None], s["mass"], torch.zeros_like(p))
    return s["mass"].copy_(torch.where(at < s["lens"][:, None, None], before + p, s["mass"]))


def _evict(s):
    c, mass, lens, table, free = s["case"], s["mass"], s["lens"].long(), s["table"], s["free"]
    B, h, S = mass.shape
    keep, recent, dev = c["keep"], c["recent"], mass.device
    D = s["data"].shape[-1] // 128
    at = torch.arange(S, device=dev)
    over = lens > keep
    key = torch.where(at < lens[:, None, None], mass, torch.full_like(mass, -math.inf))
    key = torch.where((at >= lens[:, None, None] - recent) & (at < lens[:, None, None]), torch.full_like(mass, math.inf), key)
    pick = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    i = torch.arange(keep, device=dev)
    pick = torch.nn.functional.pad(pick, (0, keep - pick.shape[-1]), value=S)
    pick = torch.where(i < lens.clamp(max=keep)[:, None, None], pick, torch.full_like(pick, S))
    pick = torch.sort(pick, -1).values
    s["kept"].copy_(torch.where(pick < S, pick, torch.full_like(pick, -1)))
    s["new_lens"].copy_(lens.clamp(max=keep))
    need = over * _pages(keep)
    base = torch.cumsum(need, 0) - need
    p = torch.arange(table.shape[1], device=dev)
    fresh = torch.where(p < _pages(keep), free[(base[:, None] + p).clamp(max=len(free) - 1)], torch.full_like(table, -1))
    s["new_table"].copy_(torch.where(over[:, None], fresh, table))
    s["taken"].copy_(need.sum().view(1))
    got = torch.gather(mass, -1, pick.clamp(max=S - 1))
    s["new_mass"].copy_(torch.where(pick < S, got, s["new_mass"]))
    # the kept tokens of the sequences over their budget, in whole pages
    rows = torch.nonzero(over).squeeze(1)
    n = _pages(keep)
    src = torch.nn.functional.pad(pick[rows], (0, n * PAGE - keep), value=S)
    some = src < S
    src = src.clamp(max=S - 1)
    page = table[rows][:, None].expand(-1, h, -1).gather(-1, src // PAGE).long()
    head = torch.arange(h, device=dev)[None, :, None]
    to = s["new_table"][rows, :n].long()
    tok = src % PAGE
    ch = torch.arange(D, device=dev)
    kbyte = (tok // 16 * (16 * D) + tok % 16 * 16)[..., None] + ch // 64 * 1024 + ch % 32 // 8 * 256 + ch // 32 % 2 * 8 + ch % 8
    vbyte = 64 * D + ch // 16 * 1024 + ch % 16 * 16 + (tok % 16 // 4 * 256 + tok // 16 * 4 + tok % 4)[..., None]
    old = _by_token(s["data"][to].flatten(0, 1), D)
    result, exps = [], []
    for part, byte in ((0, kbyte), (1, vbyte)):
        q = s["data"][page[..., None], head[..., None], byte].int() - 128  # [rows, h, n 64, D]
        e = torch.where(some, s["exps"][page, head, part * 4 + tok // BLOCK].int(), torch.full_like(src, -128).int())
        most = e.unflatten(-1, (-1, BLOCK)).amax(-1)
        q = torch.round(q * torch.ldexp(torch.ones((), device=dev), e - most.repeat_interleave(BLOCK, -1)).unsqueeze(-1)).int()
        q = q.view(len(rows), h, n, PAGE, D).transpose(1, 2)
        result.append(torch.where(some.view(len(rows), h, n, PAGE, 1).transpose(1, 2), q, old[part].view(q.shape)))
        exps.append(torch.where(most > -128, most, torch.zeros_like(most)).view(len(rows), h, n, 4).transpose(1, 2))
    written = some.view(len(rows), h, n, 4, BLOCK).any(-1).transpose(1, 2).repeat(1, 1, 1, 2)
    s["data"][to] = _by_byte(*(r.flatten(0, 1) for r in result)).view(*to.shape, h, -1)
    s["exps"][to] = torch.where(written, torch.cat(exps, -1).to(torch.int8), s["exps"][to])
    return _evicted(s)


def _evicted(s):
    return {"kept": s["kept"], "table": s["new_table"], "lens": s["new_lens"], "taken": s["taken"], "mass": s["new_mass"],
            "data": s["data"], "exponents": s["exps"]}


def run(s):
    c = s["case"]
    if own:
        import bit_weight_only_gemv_amd as B
        if c["op"] == "rotate":
            B.wq_qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], s["q_weight"], s["k_weight"], s["eps"], s["q_out"],
                              s["k_out"], neighbours=c["pairs"] == "neighbours")
            return {"q": s["q_out"], "k": s["k_out"]}
        cache = B.KV8Cache(s["data"], s["exps"])
        if c["op"] == "append":
            cache.append(s["k"], s["v"], s["slots"], s["runs"])
            return {"data": s["data"], "exponents": s["exps"]}
        if c["op"] == "evict":
            cache.evict(s["mass"], s["table"], s["lens"], c["keep"], c["recent"], s["free"], s["new_table"], s["new_lens"],
                        s["new_mass"], s["taken"], kept=s["kept"])
            return _evicted(s)
        if c["op"] == "accumulate":
            return cache.accumulate(s["q"], s["lse"], s["table"], s["lens"], s["cu"], s["held"], s["mass"], s["max_new"], s["max_len"],
                                    scale=s["scale"], window=c["window"])
        return cache.attention(s["q"], s["table"], s["lens"], s["cu"], s["max_new"], s["max_len"], scale=s["scale"],
                               window=c["window"], out=s["out"])
    return {"rotate": _rotate, "append": _append, "attend": _attend, "accumulate": _accumulate, "evict": _evict}[c["op"]](s)


# ------------------------------------------------------------ in 64 bits


def _page64(data, exps, D):
    """One head's pages, uint8 [n, 128 D], as float64 keys and values [n, 64, D], value by value from the layout's addresses."""
    dev = data.device
    t, d = torch.arange(PAGE, device=dev)[:, None], torch.arange(D, device=dev)[None, :]
    u, l = t // 16, t % 16
    kb = ((u * (D // 64) + d // 64) * 4 + d % 32 // 8) * 256 + l * 16 + d // 32 % 2 * 8 + d % 8
    vb = 64 * D + ((d // 16 * 4 + l // 4) * 16 + d % 16) * 16 + u * 4 + l % 4
    k = (data[:, kb].double() - 128) * 2.0 ** exps[:, u].double()
    v = (data[:, vb].double() - 128) * 2.0 ** exps[:, 4 + u].double()
    return k, v


def exact(case, seed):
    if case["op"] == "append":
        return None  # whole numbers alone
    if case["op"] not in ("rotate", "evict") and work(case)["bytes"] > 1.2e9:
        return None
    s = prepare(case, seed)
    if case["op"] == "rotate":
        n, pos = case["rotated"], s["positions"].double()
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * s[name + "_weight"].double()
            order = torch.arange(n, device=x.device)
            pair = order.view(2, -1) if case["pairs"] == "halves" else order.view(-1, 2).t()
            turn = torch.polar(torch.ones_like(pos[:, None]), pos[:, None] * s["freqs"])[:, None]
            z = torch.complex(x[..., pair[0]], x[..., pair[1]]) * turn
            x[..., pair[0]], x[..., pair[1]] = z.real, z.imag
            out[name] = x
        return out
    if case["op"] == "evict":
        mass = s["new_mass"].double()
        for b, n in enumerate(s["lens"].tolist()):
            for x in range(case["kv"]):
                m = s["mass"][b, x, :n].tolist()
                old = n - min(case["recent"], n)
                room = max(0, min(case["keep"], n) - (n - old))
                pick = sorted(sorted(range(old), key=lambda p: (-m[p], p))[:room]) + list(range(old, n))
                mass[b, x, :len(pick)] = torch.tensor([m[p] for p in pick], dtype=torch.float64)
        return {"kept": None, "table": None, "lens": None, "taken": None, "mass": mass, "data": None, "exponents": None}
    lens, rows = _lengths(case)
    D, h, H, w = case["dim"], case["kv"], case["heads"], case["window"]
    R, row = H // h, 0
    attend = case["op"] == "attend"
    out = torch.zeros(sum(rows), H, D, dtype=torch.float64, device="cuda") if attend else s["mass"].double()
    for b, (a, n) in enumerate(zip(lens, rows)):
        P = _pages(a)
        for x in range(h if a else 0):
            ids = s["table"][b, :P].long()
            q = s["q"][row:row + n, x * R:(x + 1) * R].double().reshape(-1, D)
            last = torch.arange(a - n, a, device="cuda").repeat_interleave(R)[:, None]
            k, v = _page64(s["data"][ids, x], s["exps"][ids, x], D)
            at = torch.arange(P * PAGE, device="cuda").view(1, -1)
            seen = (at <= last) & ((at > last - w) if w else (at >= 0))
            z = torch.matmul(q, k.view(-1, D).T.contiguous()) / math.sqrt(D)
            if attend:
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                out[row:row + n, x * R:(x + 1) * R] = torch.matmul(torch.softmax(z, -1), v.view(-1, D)).view(-1, R, D)
            else:
                lse = s["lse"][row:row + n, x * R:(x + 1) * R].double().reshape(-1, 1)
                p = torch.where(seen, torch.exp(z - lse), torch.zeros_like(z)).sum(0)[:a]
                held = int(s["held"][b])
                out[b, x, held:a] = 0
                out[b, x, :a] += p
        row += n
    return out
