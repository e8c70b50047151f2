"""8-bit key/value cache, accumulated attention weights, eviction, and the norm and
rotation of queries and keys on the GPU, against the oracle (64 bits)."""

import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_gemv_amd as B  # noqa: E402
from oracle import kv4_oracle as K4  # noqa: E402
from oracle import kv8_oracle as K8  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True, file=sys.stderr)


def ints(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


def host(t):
    """GPU tensor as numpy (float64 for floating types)."""
    return t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def f32(t):
    return t.detach().cpu().float().numpy()


def sums(n):
    return np.concatenate([[0], np.cumsum(n)])


class Made:
    """Sequences in a cache: pages shuffled, everything past a sequence's end and
    every page in no table filled with `junk` bytes (exponents too: 0x7F or 0x80 are
    none that the format has)."""

    def __init__(self, lens, H, D, seed=0, spread=1.0, extra=3, width=None, v_scale=0.7, junk=0x7F, piece=40):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens)
        need = -(-self.lens // 64)
        width = width or max(1, int(need.max()))
        self.n_pages, self.H, self.D = int(need.sum()) + extra, H, D
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), width), -1, np.int64)
        self.data = np.full((self.n_pages, H, 128 * D), junk, np.uint8)
        self.exps = np.full((self.n_pages, H, 8), junk, np.uint8).view(np.int8)
        at = 0
        for b, n in enumerate(self.lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            if n:
                k = spread * (rng.standard_normal((n, H, D)) + 2 * rng.standard_normal((1, H, D)))
                v = v_scale * rng.standard_normal((n, H, D))
                slots = self.table[b, np.arange(n) // 64] * 64 + np.arange(n) % 64
                runs = [[t, min(64 - t % 64, n - t)] for t in range(0, n, 64)]
                K8.append(self.data, self.exps, k.astype(np.float16), v.astype(np.float16), slots, runs)
        self.free = order[at:]

    def gpu(self):
        self.d, self.e = torch.from_numpy(self.data.copy()).cuda(), torch.from_numpy(self.exps.copy()).cuda()
        return B.KV8Cache(self.d, self.e)

    def same(self):
        """Whether the GPU's cache holds exactly the oracle's bytes."""
        return np.array_equal(self.d.cpu().numpy(), self.data) and np.array_equal(self.e.cpu().numpy(), self.exps)


def logit_error(D, top):
    """A logit sums D exact products (FP16 operands) whose absolute sum is `top`, in
    float32: at most D + 8 roundings, each of a whole step where a sum is cut
    (2^-23); and what its scaling, the reference and the exponential's argument add to numbers
    whose differences stay below 128 (2^-18)."""
    return (D + 8) * 2.0 ** -23 * top + 2.0 ** -18


def check_attention(out, lse, made, q, cu, scale, window=0, label=""):
    """|out - ref| <= half a step of the type, and what float32 logits and sums and the
    22-bit weights can lose.  A probability is off by its logit's error, once in itself
    and once in the sum, and by the exponential's, the weight's and the sums'
    roundings (fewer than 64 of 2^-23: 2^-17)."""
    D = made.D
    ref, lse_ref, size, top = K8.attention(made.data, made.exps, f32(q), made.table, made.lens, cu, scale, window)
    e_logit = logit_error(D, top[..., None])
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(ref) + (2 * e_logit + 2.0 ** -17) * (size + np.abs(ref)) + 2.0 ** -25
    got = host(out)
    assert np.isfinite(got).all(), label
    worst = float((np.abs(got - ref) / tol).max()) if ref.size else 0.0
    say(f"  {label}: worst |err|/bound = {worst:.4f}")
    assert worst <= 1, label
    if lse is not None:
        none = np.isinf(lse_ref)
        g = host(lse)
        assert np.array_equal(none, g == -np.inf), label
        lim = e_logit[..., 0] + 2.0 ** -17 + 2.0 ** -22 * np.abs(np.where(none, 0, lse_ref))
        assert (np.abs(np.where(none, 0, g) - np.where(none, 0, lse_ref)) <= lim).all(), label


def queries(n, heads, D, dtype, seed=1, q_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (q_scale * torch.randn(n, heads, D, generator=g)).to(dtype).cuda()


def attend(made, cache, rows, heads, dtype, seed=1, scale=None, window=0, label="", q_scale=1.0, max_rows=None,
           max_len=None):
    D = made.D
    cu = sums(rows)
    q = queries(int(cu[-1]), heads, D, dtype, seed, q_scale)
    scale = D ** -0.5 if scale is None else scale
    lse = torch.full((int(cu[-1]), heads), 7.0, device="cuda")
    out = torch.full((int(cu[-1]), heads, D), float("nan"), dtype=dtype, device="cuda")
    cache.attention(q, ints(made.table), ints(made.lens), ints(cu), max_rows if max_rows is not None else int(max(rows)),
                    max_len if max_len is not None else int(made.lens.max()), scale=scale, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    check_attention(out, lse, made, q, cu, scale, window, label)
    return q, out


# ---------------------------------------------------------------- append


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([63], [1]), ([64], [64]), ([5, 0, 31], [1, 130, 40]), ([47], [3]),
                                      ([100, 7, 0], [0, 57, 64]), ([33], [31]), ([15, 17, 30], [1, 2, 20]),
                                      ([0, 60] + [7, 15, 16, 63] * 10, [64, 70] + [1, 2, 1, 3] * 10)])
def test_append(D, dtype, lens, new):
    say("append", D, dtype, lens, new)
    H, t = 3, TYPES[dtype]
    lens, new = np.array(lens), np.array(new)
    cu = sums(new)
    made = Made(lens, H, D, seed=D + int(cu[-1]), extra=8, width=8)
    rng = np.random.default_rng(2)
    _, _, slots, runs, _ = K4.plan(lens, cu, made.table, made.free)
    T = int(cu[-1])
    # keys and values are parts of one wider buffer, of very different sizes
    qkv = torch.from_numpy(rng.standard_normal((T, 4, H, D)) * np.exp(2 * rng.standard_normal((T, 4, H, 1)))).to(t)
    cache = made.gpu()
    dev = qkv.cuda()
    cache.append(dev[:, 1], dev[:, 3], ints(slots), ints(runs))
    torch.cuda.synchronize()
    K8.append(made.data, made.exps, f32(qkv[:, 1]), f32(qkv[:, 3]), slots, runs)
    assert made.same()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_token_by_token(dtype):
    """Blocks that grow: ever larger tokens, small ones after large, and equal ones."""
    D, H, n = 64, 2, 64
    rng = np.random.default_rng(5)
    size = np.exp2(np.concatenate([np.linspace(-12, 12, 16), np.linspace(12, -12, 16), np.zeros(16),
                                   rng.integers(-8, 9, 16)]))
    x = torch.from_numpy(rng.standard_normal((2, n, H, D)) * size[:, None, None]).to(TYPES[dtype])
    made = Made([64], H, D, seed=3)
    made.data[:] = 7
    cache = made.gpu()
    dev, page = x.cuda(), int(made.table[0, 0])
    for t in range(n):
        slots = np.array([page * 64 + t])
        cache.append(dev[0, t:t + 1], dev[1, t:t + 1], ints(slots), ints([[0, 1]]))
        K8.append(made.data, made.exps, f32(x[0, t:t + 1]), f32(x[1, t:t + 1]), slots, [[0, 1]])
    torch.cuda.synchronize()
    assert made.same()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_edge_values(dtype):
    """Zeros of both signs, huge and tiny tokens, infinities and NaN, ties, the exponent's
    borders: the oracle's bytes."""
    D, H, T = 64, 1, 64
    rng = np.random.default_rng(4)
    x = rng.standard_normal((T, H, D))
    x[0:16] = 0.0
    x[3], x[5, 0, ::2] = -0.0, -0.0
    x[16:32] *= 1e-7
    x[17, 0, 5], x[18, 0, 6] = np.nan, 127.5 * 2.0 ** -20
    x[32:48] = np.round(x[32:48] * 8) / 2                     # ties
    x[40, 0, 0] = 63.5
    x[48:] *= 1e4
    x[50, 0, 1], x[51, 0, 2], x[52, 0, 3] = np.inf, -np.inf, np.nan
    x[53, 0, 4] = 65504.0
    v = torch.from_numpy(x).to(TYPES[dtype])
    made = Made([64], H, D, seed=9)
    cache = made.gpu()
    slots = np.arange(T) + 64 * made.table[0, 0]
    cache.append(v.cuda(), v.cuda().flip(0), ints(slots), ints([[0, 64]]))
    torch.cuda.synchronize()
    K8.append(made.data, made.exps, f32(v), f32(v.flip(0)), slots, [[0, 64]])
    assert made.same()
    for t in (20, 36, 53):                                    # and one at a time
        cache.append(v[t:t + 1].cuda(), v[t + 1:t + 2].cuda(), ints([slots[60]]), ints([[0, 1]]))
        K8.append(made.data, made.exps, f32(v[t:t + 1]), f32(v[t + 1:t + 2]), [slots[60]], [[0, 1]])
    torch.cuda.synchronize()
    assert made.same()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("exp", [-26, -20, -7, 0, 5, 9])
def test_append_at_the_exponents_borders(dtype, exp):
    """Blocks whose largest value stands next to 127.5 2^e, on both sides."""
    step = 2.0 ** -10 if dtype == "f16" else 2.0 ** -7
    top = 127.5 * 2.0 ** exp * (1 + step * np.array([-2, -1, 0, 1]))
    x = np.full((64, 1, 64), 0.3 * 2.0 ** exp)
    x[::16, 0, 9] = top
    v = torch.from_numpy(x).to(TYPES[dtype])
    made = Made([64], 1, 64)
    cache = made.gpu()
    slots = np.arange(64) + 64 * made.table[0, 0]
    cache.append(v.cuda(), (-v).cuda(), ints(slots), ints([[0, 64]]))
    K8.append(made.data, made.exps, f32(v), f32(-v), slots, [[0, 64]])
    assert made.same()


def test_append_skips_bad_runs_and_pages():
    D, H = 64, 2
    made = Made([64, 64], H, D)
    cache = made.gpu()
    x = torch.randn(70, H, D, generator=torch.Generator().manual_seed(0)).half().cuda()
    slots = np.concatenate([np.arange(60), np.arange(10)])
    bad = [[-1, 0], [0, 65], [69, 2], [0, 0], [5, -3], [55, 10], [1 << 30, 4], [70, 1]]
    cache.append(x, x, ints(slots), ints(bad))
    cache.append(x, x, ints(np.full(70, -1)), ints([[0, 1], [3, 2]]))
    cache.append(x, x, ints(np.arange(70) + made.n_pages * 64), ints([[0, 1], [3, 2]]))
    cache.append(x, x, ints(np.arange(70) + 60), ints([[0, 8]]))          # crosses a page's end
    torch.cuda.synchronize()
    assert made.same()


# ------------------------------------------------------------- attention


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17, 33], [64, 65, 0, 500], [1500, 3]])
def test_attention_one_row(D, dtype, lens):
    say("attention", D, dtype, lens)
    made = Made(lens, 2, D, seed=len(lens), junk=0x80 if D == 64 else 0x7F)
    attend(made, made.gpu(), [1] * len(lens), 8, TYPES[dtype], label=f"{D} {dtype} {lens}")


@pytest.mark.parametrize("H,heads", [(1, 1), (1, 16), (2, 2), (2, 10), (1, 17), (3, 21), (2, 64), (1, 40)])
def test_attention_head_groups(H, heads):
    made = Made([200, 77], H, 128, seed=heads)
    attend(made, made.gpu(), [1, 3], heads, torch.float16, label=f"{heads} heads over {H}")


@pytest.mark.parametrize("D,heads", [(64, 6), (128, 8), (256, 2)])
@pytest.mark.parametrize("lens,rows", [([40], [40]), ([130, 64, 300], [7, 64, 33]), ([700, 9], [100, 1]),
                                       ([50, 20], [0, 20]), ([5, 70], [9, 70])])
def test_attention_rows(D, heads, lens, rows):
    """Prompts and pieces of prompts; in the last, rows before the first token."""
    made = Made(lens, 2, D, seed=D)
    for dtype in TYPES.values():
        attend(made, made.gpu(), rows, heads, dtype, label=f"{D} {lens} {rows}")


@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 200, 5000, 1 << 40])
def test_attention_window(window):
    made = Made([333, 64, 1], 2, 128, seed=3)
    attend(made, made.gpu(), [20, 1, 1], 4, torch.float16, window=window, label=f"window {window}")


def test_attention_hints_do_not_change_what_is_seen():
    made = Made([900, 130], 2, 64, seed=6)
    cache = made.gpu()
    for max_rows, max_len in ((1, 1), (0, 0), (500, 1 << 20), (1, 900), (40, 64)):
        attend(made, cache, [1, 40], 4, torch.float16, max_rows=max_rows, max_len=max_len,
               label=f"hints {max_rows} {max_len}")


@pytest.mark.parametrize("n", [64, 65, 130])
def test_many_sequences(n):
    """Up to 64 sequences are taken by length, more as they come."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 300, n)
    lens[3] = lens[5]
    made = Made(lens, 2, 64, seed=n)
    cache = made.gpu()
    attend(made, cache, [1] * n, 4, torch.float16, label=f"{n} sequences")
    rows = [int(rng.integers(0, 30)) for _ in range(n)]
    attend(made, cache, rows, 4, torch.float16, label=f"{n} sequences of several rows")
    weigh(made, cache, rows, 4, torch.float16, label=f"{n} sequences of several rows")
    weigh(made, cache, [1] * n, 4, torch.float16, label=f"{n} sequences")


def test_attention_extreme_logits_and_values():
    for q_scale, v_scale, spread in ((30.0, 1.0, 3.0), (1e-4, 1e-3, 1.0), (1.0, 8000.0, 1.0), (1000.0, 0.01, 30.0),
                                     (1.0, 1e-6, 1.0)):
        made = Made([300, 2000], 1, 128, seed=8, spread=spread, v_scale=v_scale)
        for dtype in TYPES.values():
            attend(made, made.gpu(), [1, 2], 4, dtype, q_scale=q_scale, label=f"q {q_scale} v {v_scale} k {spread}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [[1, 1], [3, 50]])
def test_attention_of_logits_that_are_large_and_exact(D, dtype, rows):
    """Logits of up to 2^16 that float32 sums hold exactly: whole queries and keys, a scale that is a
    power of two.  In every sequence tokens far apart share the highest logit, in pages of lower and of
    higher ones than before, and all others are 64 or more below; so the result is nearly the mean of the
    shared ones' values, whatever the logits' size, and wrong if any step of the running reference is."""
    H, heads, t = 2, 8, TYPES[dtype]
    made = Made([1100, 700], H, D, seed=D, v_scale=0.5)
    rng, scale = np.random.default_rng(D), 2.0 ** -3
    sign = rng.choice([-1.0, 1.0], (1, 1, D))
    # q . k = 8 logit for keys `a` of size and sign[:, :, :a] of the query's 32 sign
    shared = {0: (5, 70, 300, 1040), 1: (0, 63, 64, 512)}
    for b, n in enumerate(made.lens):
        size = rng.integers(1, 40, n)                       # pages of many heights
        size[100:164] = 100                                 # one that passes all before it
        size[list(shared[b])] = 127
        k = np.where(np.arange(D) < D // 2, size[:, None, None], 0) * sign
        v = 0.5 * rng.standard_normal((n, H, D))
        slots = made.table[b, np.arange(n) // 64] * 64 + np.arange(n) % 64
        K8.append(made.data, made.exps, np.broadcast_to(k, (n, H, D)).astype(np.float16), v.astype(np.float16), slots,
                  [[j, min(64 - j % 64, n - j)] for j in range(0, n, 64)])
        blocks = K8.read_page(made.data[made.table[b, 0], 0], made.exps[made.table[b, 0], 0], D)[0]
        assert np.array_equal(blocks, k[:64, 0])            # held exactly
    cu = sums(rows)
    factor = torch.tensor([1.0, 4.0, 8.0, 32.0] * 2)[:, None]
    q = (torch.from_numpy(sign).float() * factor).expand(int(cu[-1]), heads, D).to(t).cuda()
    lse = torch.empty(int(cu[-1]), heads, device="cuda")
    cache = made.gpu()
    for max_len in (1100, 1 << 20):
        out = cache.attention(q, ints(made.table), ints(made.lens), ints(cu), max(rows), max_len, scale=scale, lse=lse)
        ref, lse_ref, size, _ = K8.attention(made.data, made.exps, f32(q), made.table, made.lens, cu, scale)
        # base-2 logits are rounded where they are scaled (twice) and taken against a reference that is
        # rounded itself when it is set, moved and shifted: at most 8 times 2^-24 of them, 2^-21 of a logit in
        # its weight's exponent.  All weights but the shared tokens' are below exp(-64)
        logit = 127 * D // 2 * scale * host(factor)[:, 0]
        assert (logit * 27 / 127 >= 64).all()
        e = 2.0 ** -21 * logit[None, :, None] + 2.0 ** -18
        tol = torch.finfo(t).eps / 2 * np.abs(ref) + 2 * e * (size + np.abs(ref)) + 2.0 ** -25
        assert (np.abs(ref) > 2 * tol).any(-1).all()        # zeros would not pass
        worst = float((np.abs(host(out) - ref) / tol).max())
        say(f"  exact logits {D} {dtype} {rows} {max_len}: worst |err|/bound = {worst:.4f}")
        assert worst <= 1
        assert (np.abs(host(lse) - lse_ref) <= e[..., 0] + 2.0 ** -17 + 2.0 ** -22 * np.abs(lse_ref)).all()
        for b in range(2):                                  # what the sequences' last rows see
            want = np.mean([made_values(made, b, j) for j in shared[b]], 0)
            assert np.abs(ref[cu[b + 1] - 1] - np.repeat(want, heads // H, 0)).max() < 1e-12


def made_values(made, b, t):
    """The values that a cached token stands for: [H, D]."""
    p = made.table[b, t // 64]
    return np.stack([K8.read_page(made.data[p, h], made.exps[p, h], made.D)[1][t % 64] for h in range(made.H)])


def test_attention_blocks_of_very_different_sizes():
    """Values of 6e4 in some blocks and 1e-6 in others, zeros, and a strong token in a
    block of zeros: weights carry the blocks' exponents, and nothing overflows."""
    D = 64
    made = Made([640], 1, D, seed=5, v_scale=0.01)
    rng = np.random.default_rng(7)
    for block, size in ((0, 6e4), (3, 1e-6), (9, 0.0), (17, 3e4), (39, 0.0)):
        k = (0.5 * rng.standard_normal((16, 1, D))).astype(np.float16)
        v = (size * (2 * rng.random((16, 1, D)) - 1)).astype(np.float16)
        if block == 9:
            k[3] = 4.0
        slots = made.table[0, block // 4] * 64 + block % 4 * 16 + np.arange(16)
        K8.append(made.data, made.exps, k, v, slots, [[0, 16]])
    for dtype in TYPES.values():
        attend(made, made.gpu(), [1], 2, dtype, label="large and small blocks")
        for q_scale in (0.01, 5.0):
            attend(made, made.gpu(), [3], 2, dtype, q_scale=q_scale, label=f"large and small blocks, q {q_scale}")


def test_attention_flat_tail_behind_a_strong_token():
    tail = Made([20000], 1, 64, seed=7, spread=0.01, v_scale=0.02)
    k = np.full((1, 1, 64), 2.0, np.float16)
    K8.append(tail.data, tail.exps, k, np.zeros((1, 1, 64), np.float16), [64 * tail.table[0, 3] + 7], [[0, 1]])
    cache = tail.gpu()
    for dtype in TYPES.values():
        q = torch.full((1, 2, 64), 0.9, dtype=dtype, device="cuda")
        lse = torch.empty(1, 2, device="cuda")
        out = cache.attention(q, ints(tail.table), ints(tail.lens), ints([0, 1]), 1, 20000, scale=0.1, lse=lse)
        check_attention(out, lse, tail, q, np.array([0, 1]), 0.1, label="flat tail")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q", [0.5, 1.0, 1.5, 2.0, 2.5])
def test_attention_beside_a_strong_token_without_values(dtype, q):
    """One page, whose strong token has values of zero: what the others give is all there is.  Their
    weights are off by a step of 2^-24, where the largest weight times 2^e of a row's first page stands at
    2^10: by 2^-34 of that."""
    D, n = 64, 64
    made = Made([n], 1, D, seed=3)
    rng = np.random.default_rng(1)
    k, v = 0.05 * rng.standard_normal((n, 1, D)), 300.0 * rng.standard_normal((n, 1, D))
    k[5], v[5] = 1.0, 0.0
    K8.append(made.data, made.exps, k.astype(np.float16), v.astype(np.float16), made.table[0, 0] * 64 + np.arange(n), [[0, n]])
    x = torch.full((1, 2, D), q, dtype=TYPES[dtype], device="cuda")
    out = host(made.gpu().attention(x, ints(made.table), ints([n]), ints([0, 1]), 1, n, scale=0.125))[0]
    keys, values = K8.read_page(made.data[made.table[0, 0], 0], made.exps[made.table[0, 0], 0], D)
    z = 0.125 * q * keys.sum(-1)
    p = np.exp(z - z.max())
    p /= p.sum()
    unit = np.repeat(2.0 ** made.exps[made.table[0, 0], 0, 4:].astype(float), 16)
    ref, size = p @ values, p @ np.abs(values)
    e = logit_error(D, 0.125 * q * np.abs(keys).sum(-1).max())
    step = 2.0 ** -34 * (p * unit).max() * (np.abs(values) / unit[:, None]).sum(0)
    tol = torch.finfo(TYPES[dtype]).eps / 2 * np.abs(ref) + (2 * e + 2.0 ** -17) * (size + np.abs(ref)) + step + \
        (2.0 ** -25 if dtype == "f16" else 0)
    assert (np.abs(ref) > 4 * tol).mean() > 0.3             # zeros would not pass
    worst = float((np.abs(out - ref) / tol).max())
    say(f"  beside a strong token, q {q}: p from {p.min():.1e}, worst |err|/bound = {worst:.4f}")
    assert worst <= 1


def test_attention_bf16_queries_of_any_size():
    made = Made([100], 1, 64, seed=2)
    for big in (1e30, 1e-30):
        attend(made, made.gpu(), [1], 2, torch.bfloat16, q_scale=big, scale=0.125 / big, label=f"q {big}")


def test_attention_skips_bad_pages():
    made = Made([300, 300], 2, 64, seed=1)
    made.table[0, 1], made.table[1, 0], made.table[1, 4] = -1, made.n_pages, 1 << 30
    attend(made, made.gpu(), [1, 2], 4, torch.float16, label="bad pages")
    made.table[:] = -5
    attend(made, made.gpu(), [1, 2], 4, torch.float16, label="no pages")


def test_attention_strided_queries():
    made = Made([90, 10], 2, 128, seed=1)
    cache = made.gpu()
    wide = torch.randn(2, 3, 12, 128, generator=torch.Generator().manual_seed(3)).half().cuda()
    cu = np.array([0, 1, 2])
    for q in (wide[:, 1, 4:12], wide[:, 2, ::3], wide[:, 0].transpose(0, 1)[:8:4].transpose(0, 1)):
        lse = torch.empty(2, q.shape[1], device="cuda")
        out = cache.attention(q, ints(made.table), ints(made.lens), ints(cu), 1, 90, lse=lse)
        check_attention(out, lse, made, q, cu, 128 ** -0.5, label=f"strides {q.stride()}")


def test_attention_is_reproducible():
    made = Made([3000, 100], 2, 128, seed=12)
    cache = made.gpu()
    a = [attend(made, cache, [1, 5], 8, torch.float16)[1] for _ in range(3)]
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


@pytest.mark.parametrize("rows", [[1, 1], [3, 70]])
def test_attention_nan_query_stays_in_its_row(rows):
    made = Made([300, 200], 2, 64, seed=4)
    cache = made.gpu()
    q = queries(sum(rows), 8, 64, torch.float16)
    cu = sums(rows)
    args = (ints(made.table), ints(made.lens), ints(cu), max(rows), 300)
    a = cache.attention(q, *args)
    q[0, 3, 5], q[1, 2, 7] = float("nan"), float("inf")
    b = cache.attention(q, *args)
    bad = torch.zeros(sum(rows), 8, dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 2] = True
    assert torch.equal(a[~bad], b[~bad]) and b[0, 3].isnan().all()


def test_attention_batches_without_rows():
    made = Made([70], 1, 64)
    cache = made.gpu()
    q = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda")
    assert cache.attention(q, ints(made.table), ints([70]), ints([0, 0]), 0, 70).shape == q.shape
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cache.attention(q, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), none, ints([0]), 0, 0)


@pytest.mark.parametrize("lens,rows,pad", [([3000, 700], [1, 1], 3), ([2500, 90], [40, 90], 7), ([90], [1], 2), ([5000], [0], 4)])
def test_padded_batches_leave_the_rows_behind_as_they_were(lens, rows, pad):
    """cu_rows ends before the rows do, in one launch and in splits that are joined."""
    made = Made(lens, 2, 64, seed=4)
    cache = made.gpu()
    n, cu = sum(rows), sums(rows)
    q = queries(n + pad, 8, 64, torch.float16)
    q[n:] = float("nan")
    args = (ints(made.table), ints(made.lens), ints(cu))
    for max_rows, max_len in ((max(max(rows), 1), max(lens)), (n + pad, 1 << 20), (1, 64)):
        out, lse = torch.full_like(q, 3.0), torch.full((n + pad, 8), 5.0, device="cuda")
        cache.attention(q, *args, max_rows, max_len, out=out, lse=lse)
        torch.cuda.synchronize()
        check_attention(out[:n], lse[:n], made, q[:n], cu, 0.125, label=f"padded {lens} {max_rows} {max_len}")
        assert (out[n:] == 3).all() and (lse[n:] == 5).all()
        lse[n:] = 1.0
        before = torch.rand(len(lens), 2, 5056, generator=torch.Generator().manual_seed(1)).cuda()
        mass, held = before.clone(), np.maximum(made.lens - np.asarray(rows), 0)
        cache.accumulate(q, lse, *args, ints(held), mass, max_rows, max_len)
        check_mass(made, q[:n], lse[:n], cu, held, host(before), mass, 0.125, label="padded masses")


def test_any_cu_rows_and_lengths_stay_in_bounds():
    """Outputs are whatever they are; rows of no sequence stay as they were."""
    made = Made([100, 130], 2, 64, seed=3)
    cache = made.gpu()
    q = queries(6, 4, 64, torch.float16)
    big = 2 ** 31 - 1
    for cu, lens in (([5, 3, 6], [100, 130]), ([-9, 2, 90], [100, 130]), ([0, big, -big - 1], [100, 130]),
                     ([0, 3, 6], [big, -7]), ([0, 2, 2], [100, 130]), ([3, 3, 3], [big, big])):
        out, lse = torch.full_like(q, 3.0), torch.full((6, 4), 3.0, device="cuda")
        mass = torch.full((2, 2, 130), 3.0, device="cuda")
        for max_rows in (1, 6):
            cache.attention(q, ints(made.table), ints(lens), ints(cu), max_rows, 130, out=out, lse=lse)
            cache.accumulate(q, lse, ints(made.table), ints(lens), ints(cu), ints([5, -1]), mass, max_rows, 130)
        torch.cuda.synchronize()
        if cu == [0, 2, 2]:
            assert (out[2:] == 3).all() and (lse[2:] == 3).all()


# ------------------------------------------------------------ accumulate


def check_mass(made, q, lse, cu, held, before, got, scale, window=0, label=""):
    """Each weight is off by its logit's error, and by the roundings of the exponent's
    argument (2^-23 of the logit and the lse), of the exponential and of the sums,
    (2^-23 of the sum for each of its terms)."""
    ref, top, count = K8.accumulate(made.data, made.exps, f32(q), f32(lse), made.table, made.lens, cu, held, before, scale, window)
    finite = np.where(np.isfinite(f32(lse)), np.abs(f32(lse)), 0)
    e = logit_error(made.D, top) + 2.0 ** -22 * (top + finite.max(initial=0)) + (count + 16) * 2.0 ** -23
    tol = e * np.abs(ref) + 2.0 ** -40
    worst = float((np.abs(host(got) - ref) / tol).max())
    say(f"  {label}: worst |err|/bound = {worst:.4f}")
    assert worst <= 1, label


def weigh(made, cache, rows, heads, dtype, held=None, scale=None, window=0, label="", max_rows=None, max_len=None,
          tokens=None, spoil=False, seed=1, q_scale=1.0):
    D = made.D
    cu = sums(rows)
    T, n = int(cu[-1]), len(made.lens)
    q = queries(T, heads, D, dtype, seed, q_scale)
    scale = D ** -0.5 if scale is None else scale
    lse = torch.empty(T, heads, device="cuda")
    args = (ints(made.table), ints(made.lens), ints(cu))
    hints = (max_rows if max_rows is not None else int(max(rows)), max_len if max_len is not None else int(made.lens.max()))
    cache.attention(q, *args, *hints, scale=scale, window=window, lse=lse)
    if spoil:
        lse[0, 0], lse[-1, -1], q[-1, -1] = float("nan"), float("inf"), float("nan")
    held = np.maximum(made.lens - np.asarray(rows), 0) if held is None else np.asarray(held)
    tokens = tokens or made.table.shape[1] * 64
    before = (torch.rand(n, made.H, tokens, generator=torch.Generator().manual_seed(3)) * 3).cuda()
    mass = before.clone()
    assert cache.accumulate(q, lse, *args, ints(held), mass, *hints, scale=scale, window=window) is mass
    torch.cuda.synchronize()
    check_mass(made, q, lse, cu, held, host(before), mass, scale, window, label)
    past = np.arange(tokens) >= made.lens[:, None]
    assert np.array_equal(host(mass).swapaxes(1, 2)[past], host(before).swapaxes(1, 2)[past])    # left as it was
    return q, lse, mass


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,rows", [([1], [1]), ([15, 16, 17, 0], [1, 1, 1, 1]), ([500, 64], [1, 3]),
                                       ([130, 70], [130, 7]), ([700, 9, 300], [100, 1, 0])])
def test_accumulate(D, dtype, lens, rows):
    say("accumulate", D, dtype, lens, rows)
    made = Made(lens, 2, D, seed=len(lens))
    weigh(made, made.gpu(), rows, 8, TYPES[dtype], label=f"{D} {dtype} {lens} {rows}")


@pytest.mark.parametrize("H,heads", [(1, 1), (2, 10), (1, 17), (3, 21), (1, 64)])
def test_accumulate_head_groups(H, heads):
    made = Made([200, 77], H, 128, seed=heads)
    weigh(made, made.gpu(), [1, 30], heads, torch.float16, label=f"{heads} heads over {H}")


@pytest.mark.parametrize("held", [[0, 0], [333, 64], [100, 70], [-5, 1 << 30]])
def test_accumulate_on_masses_that_are_held(held):
    made = Made([333, 64], 2, 64, seed=3)
    for rows in ([1, 1], [20, 64]):
        weigh(made, made.gpu(), rows, 4, torch.float16, held=held, label=f"held {held}")


@pytest.mark.parametrize("window", [1, 31, 64, 65, 5000, 1 << 40])
def test_accumulate_window(window):
    made = Made([333, 64, 1], 2, 128, seed=3)
    for rows in ([20, 1, 1], [1, 1, 1], [64, 64, 1]):
        weigh(made, made.gpu(), rows, 4, torch.float16, window=window, label=f"window {window}")


def test_accumulate_hints_sizes_and_bad_pages():
    made = Made([900, 130], 2, 64, seed=6)
    cache = made.gpu()
    for max_rows, max_len in ((1, 1), (0, 0), (500, 1 << 20), (1, 900), (40, 64)):
        weigh(made, cache, [1, 40], 4, torch.float16, max_rows=max_rows, max_len=max_len, label=f"hints {max_rows} {max_len}")
    for tokens in (1, 63, 100, 129, 2000):
        weigh(made, cache, [1, 40], 4, torch.bfloat16, tokens=tokens, label=f"{tokens} tokens")
    made.table[0, 1], made.table[1, 0], made.table[0, 4] = -1, made.n_pages, 1 << 30
    for rows in ([1, 1], [9, 60]):
        weigh(made, cache, rows, 4, torch.float16, label="bad pages")


@pytest.mark.parametrize("rows", [[1, 1], [70, 20]])
def test_accumulate_leaves_out_what_is_not_finite(rows):
    made = Made([200, 130], 2, 64, seed=6)
    q, lse, mass = weigh(made, made.gpu(), rows, 4, torch.float16, spoil=True, label="not finite")
    assert mass.isfinite().all()


def test_accumulate_of_large_logits():
    made = Made([300, 2000], 1, 128, seed=8, spread=3.0)
    for dtype in TYPES.values():
        for rows in ([1, 2], [50, 60]):
            weigh(made, made.gpu(), rows, 4, dtype, q_scale=10.0, label="large logits")


def test_accumulate_sums_to_the_rows_and_repeats():
    """Every row and head gives one in all: a group's masses sum to its rows times heads."""
    made = Made([700, 90], 2, 128, seed=1)
    cache = made.gpu()
    for rows in ([1, 1], [150, 90]):
        a = weigh(made, cache, rows, 8, torch.float16, held=[0, 0])[2]
        total = torch.stack([a[b, :, :n].sum(-1) for b, n in enumerate(made.lens)])
        assert (total - 4 * torch.tensor(rows, device="cuda")[:, None]).abs().max() <= 2e-5 * 4 * max(rows)
        assert torch.equal(a, weigh(made, cache, rows, 8, torch.float16, held=[0, 0])[2])


@pytest.mark.parametrize("heads", [4, 80])
@pytest.mark.parametrize("window", [0, 100])
def test_accumulate_without_rows_starts_the_new_tokens(heads, window):
    """Sums over no rows are 0: tokens from `held` on start at that, whatever the buffer held, and
    the others keep their masses; with any hints, a workspace of any size, on another stream and in a graph."""
    made = Made([333, 64, 0, 130], 2, 64, seed=3)
    cache, held = made.gpu(), np.array([100, 64, 0, -3])
    args = (ints(made.table), ints(made.lens), ints(np.zeros(5)), ints(held))
    q = torch.zeros(0, heads, 64, dtype=torch.float16, device="cuda")
    lse = torch.zeros(0, heads, device="cuda")
    before = torch.rand(4, 2, 400, generator=torch.Generator().manual_seed(1)).cuda()
    before[0, 0, 150:170], before[3, 1, 5] = float("nan"), float("inf")
    want, t = before.clone(), np.arange(400)
    for b, n in enumerate(made.lens):
        want[b][:, torch.from_numpy((t >= held[b]) & (t < n)).cuda()] = 0

    def call(mass, hints=(0, 333), **kw):
        return cache.accumulate(q, lse, *args, mass, *hints, window=window, **kw)

    side = torch.cuda.Stream()
    for hints in ((0, 0), (0, 333), (1, 1 << 20), (50, 64)):
        for kw in (dict(), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(stream=side),
                   dict(stream=side.cuda_stream)):
            mass = before.clone()
            torch.cuda.synchronize()
            assert call(mass, hints, **kw) is mass
            torch.cuda.synchronize()
            assert torch.equal(mass.nan_to_num(7.0), want.nan_to_num(7.0)), (hints, kw)
    graph, mass = torch.cuda.CUDAGraph(), before.clone()
    with torch.cuda.graph(graph):
        call(mass)
    for _ in range(3):
        mass.copy_(before)
        graph.replay()
        torch.rand(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.equal(mass.nan_to_num(7.0), want.nan_to_num(7.0))


# ----------------------------------------------------------------- evict


def masses(shape, seed, ties=False):
    m = np.random.default_rng(seed).random(shape).astype(np.float32) ** 6 * 30
    return np.round(m * 2) / 2 if ties else m


def check_evict(made, cache, mass, keep, recent, free=None, extra=3, label="", lens=None):
    """Against the oracle, every byte of the cache and everything behind the results' ends."""
    say("evict", label, keep, recent)
    free = made.free if free is None else np.asarray(free)
    lens = made.lens if lens is None else np.asarray(lens)
    n, H = len(lens), made.H
    before = masses((n, H, keep + extra), 77)
    new_table, new_lens, taken = ints(np.full(made.table.shape, 9)), ints(np.full(n, 9)), ints([9])
    new_mass = torch.from_numpy(before.astype(np.float32)).cuda()
    kept = cache.evict(torch.from_numpy(mass).cuda(), ints(made.table), ints(lens), keep, recent, ints(free), new_table, new_lens,
                       new_mass, taken)
    torch.cuda.synchronize()
    ref = K8.evict(made.data, made.exps, mass, made.table, lens, keep, recent, free, before)
    for got, want in zip((kept, new_table, new_lens, new_mass, taken), ref):
        assert np.array_equal(host(got), np.asarray(want).reshape(host(got).shape), equal_nan=True), label
    assert made.same(), label
    return ref


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,keep,recent", [([100], 40, 8), ([65, 64, 300, 0], 64, 0), ([500, 130, 90], 100, 100),
                                              ([1000, 200], 333, 70), ([70, 3], 1, 0), ([70, 3], 1, 1), ([129], 128, 1)])
def test_evict(D, lens, keep, recent):
    made = Made(lens, 2, D, seed=keep, extra=20, piece=9)
    cache = made.gpu()
    mass = masses((len(lens), 2, made.table.shape[1] * 64), recent)
    check_evict(made, cache, mass, keep, recent, label=f"{D} {lens}")


def test_evict_of_ties_and_odd_masses():
    made = Made([700, 650], 2, 64, seed=2, extra=30)
    cache = made.gpu()
    mass = masses((2, 2, 704), 4, ties=True)
    check_evict(made, cache, mass, 200, 20, label="ties")
    mass[:] = 0.25
    check_evict(made, cache, mass, 200, 20, label="all equal")
    mass = masses((2, 2, 704), 5)
    mass[0, 0, :500] = np.nan
    mass[0, 1, ::3], mass[0, 1, 1::3] = -0.0, 0.0
    mass[1, 0, ::5], mass[1, 0, 1::5], mass[1, 1] = np.inf, -np.inf, -mass[1, 1]
    check_evict(made, cache, mass, 300, 31, label="odd values")


def test_evict_of_long_sequences():
    made = Made([9000, 4000], 1, 64, seed=3, extra=100)
    mass = masses((2, 1, 9000), 1)
    check_evict(made, made.gpu(), mass, 3001, 17, label="long")
    # past what the threads hold (16384), by one turn and by several of eight
    for n, keep in ((16500, 16420), (27000, 1500)):
        made = Made([n, 300], 1, 64, seed=3, extra=300)
        mass = masses((2, 1, 64 * made.table.shape[1]), 2, ties=n == 27000)
        check_evict(made, made.gpu(), mass, keep, 17, label="longer")


@pytest.mark.parametrize("pages", [64, 65, 256, 257])
def test_evict_at_the_borders_of_the_ways_to_choose(pages):
    """Tables of 4096 and 16384 tokens and one page more, full and nearly empty ones; masses that many
    tokens share."""
    n = 64 * pages
    made = Made([n, 130, n - 1], 1, 64, seed=pages, extra=2 * (n // 64), spread=0.1)
    cache = made.gpu()
    for ties in (True, False):
        check_evict(made, cache, masses((3, 1, n), pages, ties=ties), 100 + n // 3, 50, label=f"{pages} pages, ties {ties}")


def test_evict_moves_blocks_of_different_exponents():
    made = Made([256], 2, 64, seed=3, extra=9)
    rng = np.random.default_rng(1)
    for j in range(16):
        k, v = (np.exp2(rng.integers(-16, 10)) * rng.standard_normal((16, 2, 64)) for _ in range(2))
        slots = made.table[0, j // 4] * 64 + j % 4 * 16 + np.arange(16)
        K8.append(made.data, made.exps, k.astype(np.float16), v.astype(np.float16), slots, [[0, 16]])
    check_evict(made, made.gpu(), masses((1, 2, 256), 2), 150, 11, label="exponents")


def test_evict_without_enough_pages_or_masses():
    made = Made([300, 400, 350], 2, 64, seed=3, extra=3)
    cache = made.gpu()
    ref = check_evict(made, cache, masses((3, 2, 448), 2), 100, 10, label="3 pages for 6")
    assert ref[-1] == 6 and (ref[1] == -1).any()
    made = Made([300, 400, 350], 2, 64, seed=3, extra=9)
    check_evict(made, made.gpu(), masses((3, 2, 210), 2), 100, 10, label="masses of 210 tokens")
    made = Made([300, 400, 350], 2, 64, seed=3, extra=9)
    made.table[0, 2], made.table[1, 0], made.table[2, 3] = -1, 1 << 20, made.n_pages
    check_evict(made, made.gpu(), masses((3, 2, 448), 2), 200, 10, label="bad pages")
    check_evict(made, made.gpu(), masses((3, 2, 448), 2), 200, 10, free=[-1, 1 << 20, made.n_pages] * 4, label="bad fresh pages")
    check_evict(made, made.gpu(), masses((3, 2, 448), 2), 200, 10, lens=[-1, 1 << 30, 77], free=made.free, label="odd lengths")


def test_evict_of_shared_pages_leaves_the_other_sequence():
    made = Made([200, 200], 2, 64, seed=3, extra=9)
    made.table[1] = made.table[0]                     # one prompt, two sequences
    cache = made.gpu()
    old = made.data.copy()
    check_evict(made, cache, masses((2, 2, 256), 2), 90, 10, label="shared")
    assert np.array_equal(old[made.table[0]], made.data[made.table[0]])


def test_evict_of_nothing():
    made = Made([70], 1, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    kept = made.gpu().evict(torch.zeros(0, 1, 64, device="cuda"), none.view(0, 2), none, 5, 1, none, none.view(0, 2).clone(), none.clone(),
                            torch.zeros(0, 1, 5, device="cuda"), ints([0]))
    assert kept.shape == (0, 1, 5)


def test_evict_of_no_sequences_takes_no_pages():
    """Fixed buffers of a step that has no sequences left: the last step's pages are not
    taken again, eagerly or in a graph, by calls with and without free pages."""
    cache = Made([70], 1, 64).gpu()
    before = cache.data.clone(), cache.exponents.clone()
    none, taken = torch.zeros(0, dtype=torch.int32, device="cuda"), ints([77])
    masses_ = torch.zeros(0, 1, 64, device="cuda"), torch.zeros(0, 1, 5, device="cuda")
    table, new_table, new_lens = none.view(0, 2), none.view(0, 2).clone(), none.clone()
    frees = [none, ints([1, 2])]

    def call(free):
        return cache.evict(masses_[0], table, none, 5, 1, free, new_table, new_lens, masses_[1], taken)

    for free in frees:
        taken.fill_(77)
        assert call(free).shape == (0, 1, 5) and int(taken) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(frees[1])
    for i in range(3):
        taken.fill_(5 + i)
        graph.replay()
        assert int(taken) == 0
    assert torch.equal(cache.data, before[0]) and torch.equal(cache.exponents, before[1])


# ------------------------------------------------------------------ rope


def check_rope(x, out, weight, pos, f, eps, neighbours, label):
    """float32 throughout and rounded once: the norm has fewer than D + 16 roundings and
    the rotation fewer than 32, of 2^-24 of |y_a| + |y_b|."""
    D = x.shape[-1]
    ref, size = K8.norm_rope(f32(x), None if weight is None else f32(weight), pos, None if f is None else host(f), eps, neighbours)
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(ref) + (D + 48) * 2.0 ** -24 * size + (2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -130)
    worst = float((np.abs(host(out) - ref) / tol).max()) if ref.size else 0.0
    say(f"  {label}: worst |err|/bound = {worst:.4f}")
    assert worst <= 1, label


def inverse_frequencies(n, base=10000.0):
    return base ** (-torch.arange(0, 2 * n, 2, dtype=torch.float64, device="cuda") / (2 * n))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("T,H,K", [(1, 32, 8), (3, 5, 1), (70, 14, 2), (5, 1, 0), (2, 0, 3), (9, 40, 3)])
def test_norm_rope(D, dtype, neighbours, T, H, K):
    say("rope", D, dtype, neighbours, T, H, K)
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(T + H)
    x = (torch.randn(T, H + 2 * K + 1, D, generator=g) * torch.exp(torch.randn(T, H + 2 * K + 1, 1, generator=g))).to(t).cuda()
    w = (1 + 0.3 * torch.randn(2, D, generator=g)).to(t).cuda()
    pos = torch.randint(-5, 200000, (T,), generator=g).int()
    q, k = (x[:, :H] if H else None), (x[:, H:H + K] if K else None)
    for n in sorted({D // 2, D // 4, 4, 24}):
        f = inverse_frequencies(n)
        a, b = B.wq_qk_norm_rope(q, k, pos.cuda(), f, w[0] if H else None, w[1] if K else None, 1e-6, neighbours=neighbours)
        for x_, out, weight in ((q, a, w[0]), (k, b, w[1])):
            if x_ is not None:
                check_rope(x_, out, weight, pos.numpy(), f, 1e-6, neighbours, f"{D} {dtype} {neighbours} {n}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_norm_rope_parts(dtype):
    """Without weights, without the norm, without the rotation; zeros, and an eps that counts."""
    t = TYPES[dtype]
    x = torch.randn(6, 9, 128, generator=torch.Generator().manual_seed(1)).to(t).cuda()
    x[2], x[3] = 0, x[3] * 1e-3
    pos, f, w = torch.arange(6, dtype=torch.int32) * 1000, inverse_frequencies(64), torch.rand(128, generator=torch.Generator().manual_seed(2)).to(t).cuda()
    for weight, eps, freq in ((None, 1e-5, f), (None, None, f), (w, 0.5, None), (None, None, None), (w, 1e-5, f)):
        a, _ = B.wq_qk_norm_rope(x, None, None if freq is None else pos.cuda(), freq, weight, eps=eps)
        check_rope(x, a, weight, pos.numpy(), freq, eps, False, f"{weight is not None} {eps} {freq is not None}")
    a, _ = B.wq_qk_norm_rope(x, None, None, None, eps=None)
    assert torch.equal(a, x)


def test_norm_rope_of_far_positions():
    """Angles of positions up to 2^20, both ways, for inv_freq up to 1: float32 products are off by
    0.06 there."""
    pos = torch.tensor([0, 1, -1, 131071, 262143, 1 << 20, -(1 << 20), 999999], dtype=torch.int32)
    x = torch.randn(8, 2, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    f = inverse_frequencies(64, 500000.0)
    for neighbours in (False, True):
        a, _ = B.wq_qk_norm_rope(x, None, pos.cuda(), f, eps=None, neighbours=neighbours)
        check_rope(x, a, None, pos.numpy(), f, None, neighbours, "far positions")
    # whole turns: every position is one of a few angles
    turn = torch.tensor([2 * np.pi * 0.25] * 4, dtype=torch.float64, device="cuda")
    a, _ = B.wq_qk_norm_rope(x[..., :64].contiguous(), None, ints([0, 4, 8, 1 << 20, -4, 400, 1 << 10, 2]), turn, eps=None)
    assert torch.equal(a[:7], x[:7, :, :64]) and torch.equal(a[7, :, :8], -x[7, :, :8])


@pytest.mark.parametrize("neighbours", [False, True])
def test_norm_rope_sines_and_cosines_are_good_to_their_bound(neighbours):
    """At an eighth of a turn the cosine and sine of a pair of ones cancel, and what is left shows their
    errors: 2^-23 each for positions up to 2^20 and inv_freq up to 1, and the rounding to FP16
    (subnormal here: 2^-25)."""
    rng = np.random.default_rng(7)
    x = torch.ones(1, 1, 64, dtype=torch.float16, device="cuda")
    worst = 0.0
    for pos in (1 << 20, -(1 << 20), 999983, -524287, 131071, 65537, -4099, 1021, 33):
        whole = rng.integers(0, int(abs(pos) / (2 * np.pi)), 32)
        f = 2 * np.pi * (whole + 0.125 + rng.uniform(-1, 1, 32) * 2.0 ** -18) / abs(pos)
        assert f.max() <= 1
        a, _ = B.wq_qk_norm_rope(x, None, ints([pos]), torch.from_numpy(f).cuda(), eps=None, neighbours=neighbours)
        ref = K8.norm_rope(np.ones((1, 1, 64)), None, [pos], f, None, neighbours)[0]
        off = np.abs(host(a) - ref)
        tol = 2.0 ** -22 + np.maximum(2.0 ** -25, 2.0 ** -11 * np.abs(ref))
        worst = max(worst, float((off / tol).max()))
    say(f"  sines and cosines: worst |err|/bound = {worst:.4f}")
    assert worst <= 1


def test_norm_rope_in_place_and_strided():
    x = torch.randn(5, 12, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w, f = torch.rand(128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda(), inverse_frequencies(64)
    pos = ints(np.arange(5) * 7)
    q, k = x[:, :8], x[:, 8:10]
    a, b = B.wq_qk_norm_rope(q, k, pos, f, w, w)
    y = x.clone()
    out = B.wq_qk_norm_rope(y[:, :8], y[:, 8:10], pos, f, w, w, q_out=y[:, :8], k_out=y[:, 8:10])
    assert torch.equal(y[:, :8], a) and torch.equal(y[:, 8:10], b) and torch.equal(y[:, 10:], x[:, 10:])
    assert out[0].data_ptr() == y.data_ptr()
    wide = torch.zeros(3, 8, 5, 128, dtype=torch.bfloat16, device="cuda")
    to = wide[1].transpose(0, 1)                      # rows and heads swapped
    B.wq_qk_norm_rope(x.transpose(0, 1)[:8].transpose(0, 1), None, pos, f, w, q_out=to)
    assert torch.equal(to, a) and not wide[0].any() and not wide[2].any()
    with pytest.raises(B.WQError):
        B.wq_qk_norm_rope(y[:, :8], None, pos, f, q_out=y.view(-1)[:5 * 8 * 128].view(5, 8, 128))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -100, 1e-6, 2.0 ** 100])
def test_norm_rope_of_bf16_heads_of_any_size(D, eps):
    """Squares past float32's range, both ways: heads of 2^-133 to 2^127 beside ordinary ones,
    single large channels among small ones.  Scaling by powers of two adds no rounding."""
    g = torch.Generator().manual_seed(D)
    size = torch.tensor([-126, -100, -75, -64, -45, -30, 0, 30, 59, 63, 64, 100, 124], dtype=torch.float64)
    x = torch.randn(5, len(size), D, generator=g).double().clamp(-7, 7) * torch.exp2(size)[:, None]
    x[1, :, 3] *= 2.0 ** 20
    x[2, :, 5:] *= 2.0 ** -40
    x = x.clamp(-3e38, 3e38).bfloat16().cuda()
    x[3, :, :] = x[3, :, :1]
    x[4, :, 1:] = 0
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16().cuda()
    pos, f = torch.arange(5, dtype=torch.int32) * 77, inverse_frequencies(D // 2)
    for neighbours in (False, True):
        a, _ = B.wq_qk_norm_rope(x, None, pos.cuda(), f, w, eps=eps, neighbours=neighbours)
        check_rope(x, a, w, pos.numpy(), f, eps, neighbours, f"{D} {eps} {neighbours}")
        for h in range(len(size)):                  # and each beside no other
            b, _ = B.wq_qk_norm_rope(x[:, h:h + 1], None, pos.cuda(), f, w, eps=eps, neighbours=neighbours)
            assert torch.equal(b[:, 0], a[:, h])


def test_norm_rope_nan_stays_in_its_head():
    x = torch.randn(3, 9, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    pos, f = ints([1, 2, 3]), inverse_frequencies(32)
    a, _ = B.wq_qk_norm_rope(x, None, pos, f)
    x[1, 4, 7], x[2, 0, 1] = float("nan"), float("inf")
    b, _ = B.wq_qk_norm_rope(x, None, pos, f)
    bad = torch.zeros(3, 9, dtype=torch.bool, device="cuda")
    bad[1, 4] = bad[2, 0] = True
    assert torch.equal(a[~bad], b[~bad]) and b[1, 4].isnan().all()


# -------------------------------------------------------------- together


class Served:
    """A serving loop on the operators together, and the same loop on the oracle."""

    def __init__(self, seqs, H, heads, D, pages, dtype, seed=0):
        self.H, self.heads, self.D, self.dtype, self.n = H, heads, D, dtype, seqs
        width = 12
        self.cache = B.KV8Cache.empty(pages, H, D)
        self.table, self.lens = ints(np.full((seqs, width), -1)), ints(np.zeros(seqs))
        self.mass = torch.zeros(seqs, H, width * 64, device="cuda")
        self.order = np.random.default_rng(seed).permutation(pages)
        self.w = (1 + 0.2 * torch.randn(2, D, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()
        self.f = inverse_frequencies(D // 2)
        self.at = np.zeros(seqs, np.int64)              # positions count on behind an eviction
        made = object.__new__(Made)
        made.H, made.D, made.table, made.lens = H, D, host(self.table).astype(np.int64), np.zeros(seqs, np.int64)
        made.data, made.exps = np.zeros((pages, H, 128 * D), np.uint8), np.zeros((pages, H, 8), np.int8)
        made.d, made.e = self.cache.data, self.cache.exponents
        self.made = made

    def free(self):
        used = set(self.made.table.ravel().tolist())
        return np.array([p for p in self.order if p not in used])

    def step(self, new, seed):
        H, D, made = self.H, self.D, self.made
        new = np.asarray(new)
        cu, T = sums(new), int(sum(new))
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(T, self.heads + 2 * H, D, generator=g).to(self.dtype).cuda()
        pos = np.concatenate([self.at[b] + np.arange(new[b]) for b in range(self.n)])
        free, after = self.free(), ints(np.zeros(self.n))
        slots, runs, taken = ints(np.zeros(T)), ints(np.zeros((B.wq_kv4_max_runs(self.n, T), 2))), ints([0])
        B.wq_kv4_plan(self.lens, ints(cu), self.table, ints(free), after, slots, runs, taken)
        q, k = B.wq_qk_norm_rope(x[:, :self.heads], x[:, self.heads:self.heads + H], ints(pos), self.f, self.w[0], self.w[1])
        v = x[:, self.heads + H:]
        self.cache.append(k, v, slots, runs)
        lse = torch.empty(T, self.heads, device="cuda")
        hints = (int(new.max()), 64 * self.table.shape[1])
        out = self.cache.attention(q, self.table, after, ints(cu), *hints, lse=lse)
        before = host(self.mass)
        self.cache.accumulate(q, lse, self.table, after, ints(cu), self.lens, self.mass, *hints)
        torch.cuda.synchronize()
        check_rope(x[:, :self.heads], q, self.w[0], pos, self.f, 1e-6, False, "q")
        table, lens, slots_, runs_, _ = K4.plan(made.lens, cu, made.table, free)
        K8.append(made.data, made.exps, f32(k), f32(v), slots_, runs_)
        held, made.table, made.lens = made.lens, table, lens
        assert made.same() and np.array_equal(host(self.table), table) and np.array_equal(host(after), lens)
        check_attention(out, lse, made, q, cu, D ** -0.5, label=f"step {seed}")
        check_mass(made, q, lse, cu, held, before, self.mass, D ** -0.5, label=f"masses {seed}")
        self.lens, self.at = after, self.at + new

    def evict(self, keep, recent):
        made = self.made
        free = self.free()
        table, lens, mass, taken = torch.empty_like(self.table), torch.empty_like(self.lens), torch.zeros_like(self.mass), ints([0])
        before = f32(self.mass)
        self.cache.evict(self.mass, self.table, self.lens, keep, recent, ints(free), table, lens, mass, taken)
        torch.cuda.synchronize()
        ref = K8.evict(made.data, made.exps, before, made.table, made.lens, keep, recent, free, np.zeros_like(before))
        made.table, made.lens = ref[1], ref[2]
        assert made.same() and np.array_equal(host(table), ref[1]) and np.array_equal(host(lens), ref[2])
        assert np.array_equal(host(mass), ref[3])
        self.table, self.lens, self.mass = table, lens, mass


@pytest.mark.parametrize("dtype,D", [("f16", 64), ("bf16", 128)])
def test_a_serving_loop(dtype, D):
    """Prompts, decode steps, drafts of several tokens and evictions in turn."""
    s = Served(3, 2, 8, D, 40, TYPES[dtype])
    s.step([150, 3, 70], 1)
    s.step([1, 1, 1], 2)
    s.evict(100, 30)
    s.step([1, 1, 1], 3)
    s.step([4, 2, 3], 4)
    s.step([90, 200, 1], 5)
    s.evict(64, 0)
    s.step([1, 0, 1], 6)
    s.evict(64, 64)
    s.step([1, 1, 1], 7)


def test_a_captured_step_serves_growing_sequences():
    """Norm, append, attention and accumulation in one graph, replayed as lengths, tables and
    inputs change; eager work and evictions between the replays."""
    H, heads, D, n, width = 2, 8, 128, 4, 8
    cache, f = B.KV8Cache.empty(60, H, D), inverse_frequencies(D // 2)
    eager = B.KV8Cache.empty(60, H, D)
    x = torch.zeros(n, heads + 2 * H, D, dtype=torch.float16, device="cuda")
    table, free = ints(np.full((n, width), -1)), ints(np.random.default_rng(0).permutation(60))
    lens, after, cu, pos = ints(np.zeros(n)), ints(np.zeros(n)), ints(np.arange(n + 1)), ints(np.zeros(n))
    slots, runs, taken = ints(np.zeros(n)), ints(np.zeros((n, 2))), ints([0])
    out, lse, mass = (torch.zeros(n, heads, D, dtype=torch.float16, device="cuda"), torch.zeros(n, heads, device="cuda"),
                      torch.zeros(n, H, width * 64, device="cuda"))

    def step(c, out, lse, mass):
        q, k = B.wq_qk_norm_rope(x[:, :heads], x[:, heads:heads + H], pos, f)
        c.append(k, x[:, heads + H:], slots, runs)
        c.attention(q, table, after, cu, 1, width * 64, out=out, lse=lse)
        c.accumulate(q, lse, table, after, cu, lens, mass, 1, width * 64)

    other = [t.clone() for t in (out, lse, mass)]
    B.wq_kv4_plan(lens, cu, table, free, after, slots, runs, taken)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(cache, out, lse, mass)
    torch.cuda.synchronize()
    mass.zero_()
    cache.data.zero_()
    cache.exponents.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out, lse, mass)
    g = torch.Generator().manual_seed(0)
    for i in range(75):
        x.copy_(torch.randn(x.shape, generator=g).half())
        if i:
            B.wq_kv4_plan(lens, cu, table, free, after, slots, runs, taken)
        graph.replay()
        step(eager, *other)
        torch.cuda.synchronize()
        assert torch.equal(out, other[0]) and torch.equal(lse, other[1]) and torch.equal(mass, other[2]), i
        assert torch.equal(cache.data, eager.data) and torch.equal(cache.exponents, eager.exponents), i
        lens.copy_(after)
        pos += 1
        free = free[int(taken):].contiguous()
    assert int(lens.min()) == 75


def test_a_captured_piece_of_a_prompt_and_an_eviction():
    """Many rows (scaled queries, splits to be joined) and an eviction in one graph, with
    workspaces of its own; every replay equals the eager calls on the same data."""
    made = Made([900, 300], 2, 128, seed=5, extra=30)
    cache, other = made.gpu(), made.gpu()
    n, heads, keep = 60, 8, 200
    q = torch.zeros(2 * n, heads, 128, dtype=torch.bfloat16, device="cuda")
    table, lens, cu, held = ints(made.table), ints(made.lens), ints([0, n, 2 * n]), ints([0, 0])
    free = ints(made.free)

    def outputs():
        return dict(out=torch.zeros_like(q), lse=torch.zeros(2 * n, heads, device="cuda"), mass=torch.zeros(2, 2, 960, device="cuda"),
                    table=torch.zeros_like(table), lens=torch.zeros_like(lens), new=torch.zeros(2, 2, keep, device="cuda"),
                    taken=ints([0]), kept=ints(np.zeros((2, 2, keep))))

    def calls(c, o):
        for max_rows in (1, n):                        # in splits, and all rows' columns together
            c.attention(q, table, lens, cu, max_rows, 900, out=o["out"], lse=o["lse"])
        c.accumulate(q, o["lse"], table, lens, cu, held, o["mass"], n, 900)
        c.evict(o["mass"], table, lens, keep, 20, free, o["table"], o["lens"], o["new"], o["taken"], kept=o["kept"])

    a, b = outputs(), outputs()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls(cache, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(cache, a)
    for i in range(4):
        q.copy_(queries(2 * n, heads, 128, torch.bfloat16, seed=i))
        graph.replay()
        torch.cuda.synchronize()
        calls(other, b)
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], b[k]) for k in a), i
        assert torch.equal(cache.data, other.data) and torch.equal(cache.exponents, other.exponents), i
        lens.sub_(1)
        torch.rand(1 << 20, device="cuda").sum()


def test_evict_of_many_sequences():
    rng = np.random.default_rng(8)
    made = Made(rng.integers(0, 200, 90), 1, 64, seed=2, extra=170)
    check_evict(made, made.gpu(), masses((90, 1, 64 * made.table.shape[1]), 3), 70, 9, label="90 sequences")


def test_calls_on_another_stream():
    """What such a call returns and uses is memory of its own stream."""
    made = Made([3000, 500], 2, 128, seed=1, extra=60)
    cache = made.gpu()
    q = queries(2, 8, 128, torch.float16)
    args = (ints(made.table), ints(made.lens), ints([0, 1, 2]))
    mass = torch.zeros(2, 2, 3008, device="cuda")
    lse = torch.empty(2, 8, device="cuda")
    want = cache.attention(q, *args, 1, 3000, lse=lse)
    cache.accumulate(q, lse, *args, ints([0, 0]), mass, 1, 3000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, lse2, f, pos = torch.zeros_like(mass), torch.empty_like(lse), inverse_frequencies(64), ints([5, 6])
    rotated = B.wq_qk_norm_rope(q, None, pos, f)[0]
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = cache.attention(q, *args, 1, 3000, lse=lse2, stream=s)
        cache.accumulate(q, lse2, *args, ints([0, 0]), other, 1, 3000, stream=s)
        turned = B.wq_qk_norm_rope(q, None, pos, f, stream=s)[0]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and torch.equal(lse, lse2) and torch.equal(mass, other) and torch.equal(turned, rotated)


def test_a_page_past_4_gib():
    """Offsets that pass 32 bits: the last pages of a cache of 4.5 GiB."""
    D, H = 256, 8
    n_pages = (9 << 29) // (H * 128 * D)
    cache = B.KV8Cache.empty(n_pages, H, D)
    made = Made([100], H, D, seed=3)
    at = [n_pages - 1, n_pages - 2]
    cache.data[at] = torch.from_numpy(made.data[made.table[0]]).cuda()
    cache.exponents[at] = torch.from_numpy(made.exps[made.table[0]]).cuda()
    q = queries(1, 8, D, torch.float16)
    lse = torch.empty(1, 8, device="cuda")
    args = (ints([at]), ints([100]), ints([0, 1]))
    out = cache.attention(q, *args, 1, 100, lse=lse)
    check_attention(out, lse, made, q, np.array([0, 1]), D ** -0.5, label="far pages")
    mass = torch.zeros(1, H, 128, device="cuda")
    cache.accumulate(q, lse, *args, ints([0]), mass, 1, 100)
    check_mass(made, q, lse, np.array([0, 1]), [0], np.zeros((1, H, 128)), mass, D ** -0.5, label="far masses")
    x = queries(1, H, D, torch.float16, seed=4)
    cache.append(x, x, ints([at[1] * 64 + 36]), ints([[0, 1]]))
    page, exps = made.data[made.table[0, 1]].copy(), made.exps[made.table[0, 1]].copy()
    for h in range(H):
        K8.append_page(page[h], exps[h], 36, f32(x)[:, h], f32(x)[:, h])
    assert np.array_equal(cache.data[at[1]].cpu().numpy(), page) and np.array_equal(cache.exponents[at[1]].cpu().numpy(), exps)


def test_tensors_of_another_device_are_refused():
    made = Made([70], 1, 64)
    cache = made.gpu()
    q = queries(1, 2, 64, torch.float16)
    with pytest.raises(ValueError):
        cache.attention(q.cpu(), ints(made.table), ints([70]), ints([0, 1]), 1, 70)
    with pytest.raises(ValueError):
        cache.attention(q, ints(made.table), ints([70]).cpu(), ints([0, 1]), 1, 70)
    with pytest.raises(ValueError):
        B.wq_qk_norm_rope(q, None, ints([0]).cpu(), inverse_frequencies(32))


@pytest.mark.parametrize("keep", [0, 100])
def test_example_block_in_8_bits(keep):
    """The example's rotated decode steps, small, against the oracle, with evictions."""
    import os
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import kv4_decode
    D, H = 64, 2
    block = kv4_decode.Block(3, 400, hidden=512, heads=8, kv_heads=H, dim=D, bits=8, rotate=True)
    prompt = np.array([62, 200, 1])
    kv = block.fill(prompt.tolist())
    made = object.__new__(Made)
    made.H, made.D, made.d, made.e = H, D, block.cache.data, block.cache.exponents
    made.data, made.exps = np.zeros(made.d.shape, np.uint8), np.zeros(made.e.shape, np.int8)
    free = torch.randperm(len(made.data), generator=torch.Generator().manual_seed(0)).numpy()
    made.table, made.lens, slots, runs, taken = K4.plan(np.zeros(3, np.int64), sums(prompt), np.full(block.table.shape, -1), free)
    free = np.roll(free, -taken)
    K8.append(made.data, made.exps, f32(kv[0]), f32(kv[1]), slots, runs)
    step, x, proj, att, y = block.stepper(0, keep > 0)
    cu, at = np.arange(4), prompt.copy()
    g = torch.Generator().manual_seed(1)
    for i in range(5):
        if keep and i in (1, 4):
            mass = f32(block.mass)
            block.evict(keep)
            _, made.table, made.lens, want, _ = K8.evict(made.data, made.exps, mass, made.table, made.lens, keep, keep // 4, free,
                                                         np.zeros_like(mass))
            used = np.isin(free, made.table)
            free = np.concatenate([free[~used], free[used]])
            assert np.array_equal(f32(block.mass), want) and np.array_equal(host(block.free), free)
        x.copy_(torch.randn(x.shape, generator=g).half().view(torch.int16))
        step()
        torch.cuda.synchronize()
        q, k, v = block.split(proj)                    # rotated in place
        held = made.lens
        made.table, made.lens, slots, runs, taken = K4.plan(made.lens, cu, made.table, free)
        free = np.roll(free, -taken)
        at += 1
        K8.append(made.data, made.exps, f32(k), f32(v), slots, runs)
        assert made.same() and np.array_equal(host(block.lens), made.lens) and np.array_equal(host(block.table), made.table)
        assert np.array_equal(host(block.at), at)
        rms = f32(q).astype(np.float64).reshape(-1, D)
        assert np.allclose((rms ** 2).mean(-1), 1, atol=2e-3)                # normed, and turned by no length
        check_attention(att, block.lse, made, q, cu, D ** -0.5, label=f"example step {i}")
        assert torch.isfinite(y.view(torch.float16).float()).all() and (y != 0).any()
    if keep:
        assert (made.lens <= keep + 1).all() and block.mass.isfinite().all() and (block.mass > 0).any()


def test_example_runs(capsys):
    import os
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import kv4_decode
    kv4_decode.main(["--bits", "8", "--rotate", "--keep", "150", "--seqs", "3", "--prompt", "200", "--steps", "40"])
    kv4_decode.main(["--rotate", "--seqs", "2", "--prompt", "100", "--steps", "4"])
    assert capsys.readouterr().out.count("us a step") == 2
