"""4-bit key/value cache on the GPU against the oracle (64 bits)."""

import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import bit_weight_only_gemv_amd as B  # noqa: E402
from oracle import kv4_oracle as K4  # noqa: E402

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


class Made:
    """Sequences in a cache: pages shuffled, everything past a sequence's end and
    every page in no table filled with 0xFF bytes (NaN scales and offsets)."""

    def __init__(self, lens, H, D, seed=0, spread=1.0, extra=3, width=None, v_scale=0.7):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens)
        need = -(-self.lens // 64)
        width = width or max(1, int(need.max()))
        self.n_pages = int(need.sum()) + extra
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), width), -1, np.int64)
        self.data = np.full((self.n_pages, H, 80 * D), 0xFF, np.uint8)
        self.summary = np.full((self.n_pages, H, 2, D), np.nan, np.float16)
        at = 0
        for b, n in enumerate(self.lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            if n:
                k = spread * (rng.standard_normal((n, H, D)) + 2 * rng.standard_normal((1, H, D)))
                v = v_scale * rng.standard_normal((n, H, D))
                slots = self.table[b, np.arange(n) // 64] * 64 + np.arange(n) % 64
                self._append(k.astype(np.float16), v.astype(np.float16), slots)

    def _append(self, k, v, slots):
        K4.append(self.data, self.summary, k, v, slots)

    def gpu(self):
        self.d, self.s = torch.from_numpy(self.data).cuda(), torch.from_numpy(self.summary).cuda()
        return B.KV4Cache(self.d, self.s)


def check_attention(out, lse, made, q, cu, scale, window=0, sel=None, label=""):
    """|out - ref| <= half a step of the type, and what float32 logits and sums and
    the FP16 probabilities can lose.  A logit sums D products whose absolute sum
    is `top`, in float32 with fewer than 64 roundings: 64 2^-24 top.  A
    probability is off by that, once in itself and once in the sum, by the
    exponential's and the sums' roundings (fewer than 64: 2^-17), and for BF16
    outputs by one FP16 rounding (2^-11)."""
    ref, lse_ref, size, top = K4.attention(made.data, f32(q), made.table, made.lens, cu, scale, window, sel)
    bf = q.dtype == torch.bfloat16
    e_logit = 64 * 2.0 ** -24 * top[..., None] + 2.0 ** -18
    e_p = 2 * e_logit + 2.0 ** -17 + (2.0 ** -11 if bf else 0)
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(ref) + e_p * (size + np.abs(ref)) + 2.0 ** -25
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


def attend(made, cache, rows, heads, dtype, seed=1, scale=None, window=0, sel=None, label="", q_scale=1.0,
           max_rows=None, max_len=None):
    D = cache.head_dim
    cu = np.concatenate([[0], np.cumsum(rows)])
    g = torch.Generator().manual_seed(seed)
    q = (q_scale * torch.randn(int(cu[-1]), heads, D, generator=g)).to(dtype).cuda()
    scale = D ** -0.5 if scale is None else scale
    lse = torch.full((int(cu[-1]), heads), 7.0, device="cuda")
    out = torch.full((int(cu[-1]), heads, D), float("nan"), dtype=dtype, device="cuda")
    cache.attention(q, ints(made.table), ints(made.lens), ints(cu),
                    max_rows if max_rows is not None else int(max(rows)),
                    max_len if max_len is not None else int(made.lens.max()), scale=scale, window=window,
                    sel=None if sel is None else ints(sel), out=out, lse=lse)
    torch.cuda.synchronize()
    check_attention(out, lse, made, q, cu, scale, window, sel, label)
    return q, out


# ------------------------------------------------------------------ plan


@pytest.mark.parametrize("n_seqs,most_len,most_new,short", [
    (1, 1, 2, 0), (1, 500, 300, 0), (5, 200, 130, 0), (64, 300, 2, 0), (70, 200, 3, 9), (1025, 400, 40, 0),
    (2500, 300, 5, 100), (8192, 100, 3, 0)])
def test_plan(n_seqs, most_len, most_new, short):
    say("plan", n_seqs, most_len, most_new, short)
    rng = np.random.default_rng(n_seqs + most_len)
    lens = rng.integers(0, most_len, n_seqs)
    new = rng.integers(0, most_new, n_seqs)
    if n_seqs == 1:
        new[0] = most_new
    cu = np.concatenate([[0], np.cumsum(new)])
    width = int((-(-(lens + new) // 64)).max()) + 1
    held = -(-lens // 64)
    order = rng.permutation(int(held.sum()) + int((-(-(lens + new) // 64) - held).sum()) + 4)
    table = np.full((n_seqs, width), -1)
    at = 0
    for b in range(n_seqs):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = order[at:][: len(order) - at - short - 4] if short else order[at:]
    want = K4.plan(lens, cu, table, free)
    T, n_runs = int(cu[-1]), len(want[3])
    t, slots, runs = ints(table), ints(np.full(T, 9)), ints(np.full((n_runs, 2), 9))
    after, taken = ints(np.zeros(n_seqs)), ints([0])
    for _ in range(2):                          # a second call gives the same
        B.wq_kv4_plan(ints(lens), ints(cu), t, ints(free), after, slots, runs, taken)
        torch.cuda.synchronize()
        for got, ref in zip((t, after, slots, runs, taken), want):
            assert np.array_equal(host(got), np.asarray(ref).reshape(host(got).shape))


def test_plan_narrow_table():
    lens, cu = np.array([100, 0]), np.array([0, 100, 130])
    table = np.array([[5, 6], [-1, -1]])
    want = K4.plan(lens, cu, table, np.array([9, 8, 7]))
    t, slots, runs = ints(table), ints(np.zeros(130)), ints(np.zeros((len(want[3]), 2)))
    after, taken = ints([0, 0]), ints([0])
    B.wq_kv4_plan(ints(lens), ints(cu), t, ints([9, 8, 7]), after, slots, runs, taken)
    for got, ref in zip((t, after, slots, runs, taken), want):
        assert np.array_equal(host(got), np.asarray(ref).reshape(host(got).shape))
    assert (host(slots)[28:100] == -1).all()


# ---------------------------------------------------------------- append


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([63], [1]), ([64], [64]), ([5, 0, 31], [1, 130, 40]),
                                      ([100, 7, 0], [0, 57, 64]), ([33], [31])])
def test_append(D, dtype, lens, new):
    say("append", D, dtype, lens, new)
    H, t = 3, TYPES[dtype]
    lens, new = np.array(lens), np.array(new)
    cu = np.concatenate([[0], np.cumsum(new)])
    made = Made(lens, H, D, seed=D + int(cu[-1]), extra=8, width=8)
    rng = np.random.default_rng(2)
    free = np.setdiff1d(np.arange(made.n_pages), made.table)
    table, after, slots, runs, _ = K4.plan(lens, cu, made.table, free)
    T = int(cu[-1])
    # keys and values are parts of one wider buffer
    qkv = torch.from_numpy(rng.standard_normal((T, 4, H, D)) * np.exp(rng.standard_normal((T, 1, H, 1)))).to(t)
    cache = made.gpu()
    dev = qkv.cuda()
    cache.append(dev[:, 1], dev[:, 3], ints(slots), ints(runs))
    torch.cuda.synchronize()
    K4.append(made.data, made.summary, f32(qkv[:, 1]), f32(qkv[:, 3]), slots)
    assert np.array_equal(made.d.cpu().numpy(), made.data)
    assert np.array_equal(made.s.cpu().numpy(), made.summary, equal_nan=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_edge_values(dtype):
    """Constant groups, huge and tiny ranges, signed zeros, infinities and NaN:
    the cache stays finite and equal to the oracle's."""
    D, H, T = 64, 1, 64
    rng = np.random.default_rng(4)
    x = rng.standard_normal((T, H, D))
    x[0], x[1], x[2], x[3, :, ::2] = 0.0, -0.0, 3.25, -0.0
    x[4, 0, 5], x[5, 0, 6], x[6, 0, 7] = np.nan, np.inf, -np.inf
    x[7] *= 1e4
    x[8] = np.where(x[8] > 0, 6e4, -6e4)
    x[9] *= 1e-7
    x[10] = 1000 + x[10] * 1e-2
    x[11:20] = np.round(x[11:20] * 2) / 4           # many ties
    x[20] = np.nan
    v = torch.from_numpy(x).to(TYPES[dtype])
    made = Made([64], H, D, seed=9)
    cache = made.gpu()
    slots = np.arange(T) + 64 * made.table[0, 0]
    cache.append(v.cuda(), v.cuda().flip(0), ints(slots), ints([[0, 64]]))
    torch.cuda.synchronize()
    K4.append(made.data, made.summary, f32(v), f32(v.flip(0)), slots)
    assert np.array_equal(made.d.cpu().numpy(), made.data)
    assert np.array_equal(made.s.cpu().numpy().astype(np.float32), made.summary.astype(np.float32), equal_nan=True)
    k, w, _ = K4.read_page(made.data[made.table[0, 0], 0], D)
    assert np.isfinite(k).all() and np.isfinite(w).all()


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
    assert np.array_equal(made.d.cpu().numpy(), made.data)


# ------------------------------------------------------------- attention


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[1], [31, 32, 33], [64, 65, 0, 500], [1500, 3]])
def test_attention_one_row(D, dtype, lens):
    say("attention", D, dtype, lens)
    made = Made(lens, 2, D, seed=len(lens))
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


def test_attention_extreme_logits_and_values():
    for q_scale, v_scale, spread in ((30.0, 1.0, 3.0), (1e-4, 1e-3, 1.0), (1.0, 8000.0, 1.0), (1000.0, 0.01, 30.0),
                                     (1.0, 3.0, 1.0)):
        made = Made([300, 2000], 1, 128, seed=8, spread=spread, v_scale=v_scale)
        for dtype in TYPES.values():
            attend(made, made.gpu(), [1, 2], 4, dtype, q_scale=q_scale, label=f"q {q_scale} v {v_scale} k {spread}")


def test_attention_mixed_value_scales():
    """Small values first, then a page of very large ones, and a flat long tail
    beside one strong token: nothing overflows and the tail keeps its weight."""
    made = Made([3000], 1, 64, seed=5, v_scale=0.01)
    k, v = np.zeros((64, 1, 64), np.float16), np.full((64, 1, 64), 1.0, np.float16)
    v[:, 0, ::2] = 60000.0
    slots = np.arange(64) + 64 * made.table[0, 20]
    K4.append(made.data, made.summary, k, v, slots)
    attend(made, made.gpu(), [1], 2, torch.float16, label="large page")
    tail = Made([20000], 1, 64, seed=7, spread=0.01, v_scale=0.02)
    k = np.full((1, 1, 64), 2.0, np.float16)
    K4.append(tail.data, tail.summary, k, np.zeros((1, 1, 64), np.float16), [64 * tail.table[0, 3] + 7])
    cache = tail.gpu()
    q = torch.full((1, 2, 64), 0.9, dtype=torch.float16, device="cuda")
    lse = torch.empty(1, 2, device="cuda")
    out = cache.attention(q, ints(tail.table), ints(tail.lens), ints([0, 1]), 1, 20000, scale=0.1, lse=lse)
    check_attention(out, lse, tail, q, np.array([0, 1]), 0.1, label="flat tail")


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


def test_attention_nan_query_stays_in_its_row():
    made = Made([100, 100], 1, 64, seed=12)
    cache = made.gpu()
    q = torch.randn(5, 4, 64, generator=torch.Generator().manual_seed(3)).half().cuda()
    args = (ints(made.table), ints(made.lens), ints([0, 3, 5]), 3, 100)
    clean = cache.attention(q, *args)
    bad = q.clone()
    bad[1, 2, 7] = float("nan")
    out = cache.attention(bad, *args)
    assert out[1, 2].isnan().all()
    keep = torch.ones(5, 4, dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(out[keep], clean[keep])


# ---------------------------------------------------------------- select


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,rows,heads,n_sel", [([1], [1], 2, 2), ([64, 65, 0], [1, 1, 1], 2, 4),
                                                   ([3000, 900], [1, 3], 8, 7), ([9000], [2], 10, 40),
                                                   ([500, 20000], [1, 1], 4, 100)])
def test_select_and_sparse_attention(D, dtype, lens, rows, heads, n_sel):
    say("select", D, dtype, lens, rows, heads, n_sel)
    if D == 256 and max(lens) > 10000:
        lens = [500, 8000]
    made = Made(lens, 2, D, seed=n_sel)
    cache = made.gpu()
    cu = np.concatenate([[0], np.cumsum(rows)])
    g = torch.Generator().manual_seed(1)
    q = torch.randn(int(cu[-1]), heads, D, generator=g).to(TYPES[dtype]).cuda()
    args = (ints(made.table), ints(made.lens), ints(cu))
    sel = cache.select(q, *args, n_sel)
    want = K4.select(made.summary, f32(q), made.table, made.lens, cu, n_sel)
    assert np.array_equal(host(sel), want)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = cache.attention(q, *args, max(rows), max(lens), sel=sel, lse=lse)
    check_attention(out, lse, made, q, cu, D ** -0.5, 0, want, f"sparse {D} {dtype} {lens}")


def test_select_ties_go_to_the_lower_page():
    made = Made([64 * 300], 1, 64, seed=1)
    for p in range(300):
        made.summary[made.table[0, p]] = made.summary[made.table[0, p % 3]]
    cache = made.gpu()
    q = torch.randn(1, 3, 64, generator=torch.Generator().manual_seed(5)).half().cuda()
    for n in (2, 3, 50, 101, 102, 299, 300, 400):
        sel = cache.select(q, ints(made.table), ints(made.lens), ints([0, 1]), n)
        assert np.array_equal(host(sel), K4.select(made.summary, f32(q), made.table, made.lens, [0, 1], n)), n


def test_select_is_exact_where_float32_is_not():
    """Bounds that differ in the last bits of their 64-bit sums' float32 rounding."""
    made = Made([64 * 200], 1, 128, seed=2)
    rng = np.random.default_rng(0)
    base = rng.standard_normal(128).astype(np.float16)
    for p in range(200):
        s = base.copy()
        j = rng.integers(0, 128, 2)
        s[j] = np.nextafter(s[j], np.float16(9), dtype=np.float16)
        made.summary[made.table[0, p], 0] = s
    cache = made.gpu()
    q = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(5)).half().cuda()
    for n in (5, 20, 100):
        sel = cache.select(q, ints(made.table), ints(made.lens), ints([0, 1]), n)
        assert np.array_equal(host(sel), K4.select(made.summary, f32(q), made.table, made.lens, [0, 1], n)), n


def test_sparse_attention_takes_any_list():
    """A caller's own list: unused entries anywhere, pages past the row's position."""
    made = Made([700, 130], 2, 64, seed=4)
    sel = np.full((3, 2, 6), -1)
    sel[0, 0] = [-1, 3, -1, 5, 10, -1]
    sel[0, 1] = [0, 1, 2, 9, 10, 11]
    sel[1, 0] = [10, 2, 1 << 30, 7, -1, 0]
    sel[2, 0] = [0, 1, 2, 3, 4, 5]
    attend(made, made.gpu(), [2, 1], 4, torch.float16, sel=sel, label="own list")


# ------------------------------------------------- streams, graphs, steps


def step(cache, free, k, v, q, state):
    table, lens, cu, after, slots, runs, taken, sel, out, out2 = state
    B.wq_kv4_plan(lens, cu, table, free, after, slots, runs, taken)
    cache.append(k, v, slots, runs)
    cache.attention(q, table, after, cu, 1, 400, out=out)
    cache.select(q, table, after, cu, 3, sel=sel)
    cache.attention(q, table, after, cu, 1, 400, sel=sel, out=out2)


@pytest.mark.parametrize("how", ["stream", "graph"])
def test_steps_on_a_side_stream_and_in_a_graph(how):
    """Decode steps in which sequences grow over page ends; each step's cache and
    outputs against the oracle."""
    H, D, heads, n = 2, 64, 4, 3
    made = Made([62, 0, 191], H, D, seed=3, extra=40, width=6)
    cache = made.gpu()
    free_np = np.setdiff1d(np.arange(made.n_pages), made.table)
    cu = np.arange(n + 1)
    g = torch.Generator().manual_seed(0)
    k, v, q = (torch.zeros(n, c, D, dtype=torch.float16, device="cuda") for c in (H, H, heads))
    free = ints(free_np)
    state = [ints(made.table), ints(made.lens), ints(cu), ints(np.zeros(n)), ints(np.zeros(n)), ints(np.zeros((n, 2))),
             ints([0]), ints(np.zeros((n, H, 3))), torch.empty_like(q), torch.empty_like(q)]
    side = torch.cuda.Stream()
    graph = None
    if how == "graph":
        saved = [made.d.clone(), made.s.clone(), state[0].clone()]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(cache, free, k, v, q, state)          # loads the kernels
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(cache, free, k, v, q, state)
        made.d.copy_(saved[0]), made.s.copy_(saved[1]), state[0].copy_(saved[2])
    for i in range(5):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g).half())
        state[1].copy_(ints(made.lens))
        free.copy_(ints(free_np))
        torch.cuda.synchronize()
        if graph is None:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step(cache, free, k, v, q, state)
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
        torch.cuda.synchronize()
        made.table, made.lens, slots, runs, taken = K4.plan(made.lens, cu, made.table, free_np)
        free_np = np.roll(free_np, -taken)
        K4.append(made.data, made.summary, f32(k), f32(v), slots)
        assert np.array_equal(made.d.cpu().numpy(), made.data), i
        assert np.array_equal(host(state[0]), made.table), i
        check_attention(state[8], None, made, q, cu, D ** -0.5, label=f"step {i}")
        sel = K4.select(made.summary, f32(q), made.table, made.lens, cu, 3)
        assert np.array_equal(host(state[7]), sel), i
        check_attention(state[9], None, made, q, cu, D ** -0.5, 0, sel, f"step {i} sparse")


def test_explicit_stream():
    made = Made([500, 3], 2, 64, seed=3)
    cache = made.gpu()
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(0)).half().cuda()
    args = (ints(made.table), ints(made.lens), ints([0, 1, 2]), 1, 500)
    want = cache.attention(q, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        out = cache.attention(q, *args, stream=s)
        side.synchronize()
        assert torch.equal(out, want)


def test_long_cache_addresses_past_32_bits():
    """Pages whose bytes lie past 4 GiB of the cache, append and both attentions."""
    D, H, n_pages = 256, 8, 30000                   # 4.9 GB
    data = torch.zeros(n_pages, H, 80 * D, dtype=torch.uint8, device="cuda")
    summary = torch.zeros(n_pages, H, 2, D, dtype=torch.float16, device="cuda")
    cache = B.KV4Cache(data, summary)
    pages = np.array([29999, 27000, 29998])
    rng = np.random.default_rng(1)
    k, v = (torch.from_numpy(rng.standard_normal((150, H, D))).half() for _ in range(2))
    slots = pages[np.arange(150) // 64] * 64 + np.arange(150) % 64
    cache.append(k.cuda(), v.cuda(), ints(slots), ints([[0, 64], [64, 64], [128, 22]]))
    torch.cuda.synchronize()
    made = Made([0], H, D, extra=3)
    made.table, made.lens = np.array([[0, 1, 2]]), np.array([150])
    made.data[:], made.summary[:] = 0, 0
    K4.append(made.data, made.summary, f32(k), f32(v), np.arange(150))
    assert np.array_equal(data[torch.from_numpy(pages).cuda()].cpu().numpy(), made.data)
    q = torch.randn(2, 16, D, generator=torch.Generator().manual_seed(0)).half().cuda()
    args = (ints(pages[None]), ints([150]), ints([0, 2]))
    sel = cache.select(q, *args, 2)
    want = K4.select(made.summary, f32(q), made.table, made.lens, [0, 2], 2)
    assert np.array_equal(host(sel), want)
    for s, w in ((None, None), (sel, want)):
        out = cache.attention(q, *args, 2, 150, sel=s)
        check_attention(out, None, made, q, np.array([0, 2]), D ** -0.5, 0, w, "far pages")


# --------------------------------------------- many rows, memory, example


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 70])
def test_attention_two_column_tiles(D, window):
    """Rows enough for two column tiles a wave, ending inside the second or the
    first, windows, large value scales and rows before the first token."""
    for lens, rows, heads in (([300, 40], [75, 40], 2), ([130, 0], [33, 3], 4), ([90], [130], 1)):
        made = Made(lens, 1, D, seed=11, v_scale=2.0)
        for dtype in TYPES.values():
            attend(made, made.gpu(), rows, heads, dtype, window=window, label=f"{D} {rows} {heads} {window}")


def test_bad_row_tables_stay_in_bounds():
    """cu_rows that does not rise, runs past the rows or is negative, and lengths
    out of step with the table: nothing outside the given rows is written."""
    made = Made([100, 50, 200], 2, 64, seed=2)
    cache = made.gpu()
    q = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(3)).half().cuda()
    room = torch.full((10, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    for cu in ([0, 4, 2, 6], [0, 9, 12, 50], [-3, 1, 2, 6], [5, 5, 5, 5], [0, 2, 4, 6]):
        for lens in (made.lens, [1 << 30, -5, 0]):
            cache.attention(q, ints(made.table), ints(lens), ints(cu), 2, 200, out=room[2:8])
            sel = cache.select(q, ints(made.table), ints(lens), ints(cu), 2)
            cache.attention(q, ints(made.table), ints(lens), ints(cu), 2, 200, sel=sel, out=room[2:8])
            slots, runs = ints(np.zeros(6)), ints(np.zeros((6, 2)))
            B.wq_kv4_plan(ints(lens), ints(cu), ints(made.table), ints([1, 2]), ints([0, 0, 0]), slots, runs, ints([0]))
    torch.cuda.synchronize()
    assert (room[:2] == 5).all() and (room[8:] == 5).all()


def test_launch_loop_keeps_device_memory_flat():
    """The library allocates nothing: the caller's workspaces are all there is."""
    made = Made([3000, 100], 2, 128, seed=1)
    cache = made.gpu()
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(3)).half().cuda()
    args = (ints(made.table), ints(made.lens), ints([0, 1, 2]))
    out, sel = torch.empty_like(q), ints(np.zeros((2, 2, 5)))
    work = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def once():
        cache.select(q, *args, 5, sel=sel, workspace=work)
        cache.attention(q, *args, 1, 3000, out=out, workspace=work)
        cache.attention(q, *args, 1, 3000, sel=sel, out=out, workspace=work)

    for _ in range(500):
        once()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(2000):
        once()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("pages", [0, 3])
def test_example_block(pages):
    """The example's decode steps, small, against the oracle: the cache's bytes, the
    attention's output from the step's own queries, and the growing lengths."""
    import os
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import kv4_decode
    block = kv4_decode.Block(3, 400, hidden=512, heads=8, kv_heads=2, dim=64)
    prompt = [62, 200, 1]
    kv = block.fill(prompt)
    made = Made([0], 2, 64, extra=0)
    made.data, made.summary = np.zeros(block.cache.data.shape, np.uint8), np.zeros(block.cache.summary.shape, np.float16)
    made.n_pages = len(made.data)
    free = torch.randperm(made.n_pages, generator=torch.Generator().manual_seed(0)).numpy()
    made.table, made.lens, slots, _, taken = K4.plan(np.zeros(3, np.int64), np.concatenate([[0], np.cumsum(prompt)]),
                                                     np.full(block.table.shape, -1), free)
    free = np.roll(free, -taken)
    K4.append(made.data, made.summary, f32(kv[0]), f32(kv[1]), slots)
    step, x, proj, att, y = block.stepper(pages)
    cu = np.arange(4)
    g = torch.Generator().manual_seed(1)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g).half().view(torch.int16))
        step()
        torch.cuda.synchronize()
        q, k, v = block.split(proj)
        made.table, made.lens, slots, _, taken = K4.plan(made.lens, cu, made.table, free)
        free = np.roll(free, -taken)
        K4.append(made.data, made.summary, f32(k), f32(v), slots)
        assert np.array_equal(block.cache.data.cpu().numpy(), made.data), i
        assert np.array_equal(host(block.lens), made.lens) and np.array_equal(host(block.table), made.table)
        sel = K4.select(made.summary, f32(q), made.table, made.lens, cu, pages) if pages else None
        check_attention(att, None, made, q, cu, 64 ** -0.5, 0, sel, f"example step {i}")
        assert torch.isfinite(y.view(torch.float16).float()).all() and (y != 0).any()


# ------------------------------------------ softmax weights and their range


def check_held(out, made, q, cu, scale, label, sinks=0.0):
    """check_attention's bound with nothing for the weights' own rounding, in either
    type: weights are held in 22 bits or more, which 2^-17 covers with room.  sinks:
    absolute error allowed, as the caller derives it."""
    ref, _, size, top = K4.attention(made.data, f32(q), made.table, made.lens, cu, scale)
    e_p = 2 * (64 * 2.0 ** -24 * top[..., None] + 2.0 ** -18) + 2.0 ** -17
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(ref) + e_p * (size + np.abs(ref)) + 2.0 ** -25 + sinks
    worst = float((np.abs(host(out) - ref) / tol).max())
    say(f"  {label}: worst |err|/bound = {worst:.4f}")
    assert worst <= 1, label


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[2, 3, 5], [64, 70], [1000]])
def test_attention_weights_keep_their_bits(D, dtype, lens):
    """Few values of both signs nearly cancel, and what a weight lost by a rounding
    to 11 bits would show beside the small result."""
    made = Made(lens, 2, D, seed=21, v_scale=1.0)
    n = len(lens)
    q = torch.randn(n, 16, D, generator=torch.Generator().manual_seed(4)).to(TYPES[dtype]).cuda()
    out = made.gpu().attention(q, ints(made.table), ints(made.lens), ints(np.arange(n + 1)), 1, max(lens), scale=0.02)
    check_held(out, made, q, np.arange(n + 1), 0.02, f"{D} {dtype} {lens}")


class Tail(Made):
    """Flat logits and values of one sign, behind one strong token of zero values in
    each of the first `sinks` pages: the small weights make up the whole result."""

    def __init__(self, n, D, nats, big=0.0, sinks=8, seed=7):
        self.big = big
        super().__init__([n], 1, D, seed=seed, spread=0.01, v_scale=0.02)
        k, v = np.full((1, 1, D), 2.0, np.float16), np.zeros((1, 1, D), np.float16)
        for p in range(sinks):
            K4.append(self.data, self.summary, k, v, [64 * self.table[0, p] + 5 * p])
        self.scale = nats / (2.0 * D)

    def _append(self, k, v, slots):
        v = v + np.float16(0.05)
        if self.big:
            v[..., :32] = v[..., :32].astype(np.float32) * (self.big / 0.05)
        super()._append(k, v, slots)

    def check(self, dtype, max_len, label):
        D = self.data.shape[2] // 80
        q = torch.ones(1, 2, D, dtype=dtype, device="cuda")
        out = self.gpu().attention(q, ints(self.table), ints(self.lens), ints([0, 1]), 1, max_len, scale=self.scale)
        # a weight loses at most 2^-25 of what stands for 2^8 or more at the sinks: 64
        # tokens of their pages, values below 0.14 (or big's)
        sinks = np.full(D, 64 * 2.0 ** -33 * 0.14)
        sinks[:32] *= max(1.0, self.big / 0.05)
        check_held(out, self, q, np.array([0, 1]), self.scale, label, sinks)


@pytest.mark.parametrize("D,n", [(64, 20000), (128, 9000), (256, 5000)])
@pytest.mark.parametrize("nats", [11, 13, 15, 17])
def test_attention_keeps_small_weights(D, n, nats):
    """The whole cache in one workgroup, and split as for its length."""
    made = Tail(n, D, nats)
    for dtype in TYPES.values():
        for max_len in (1, n):
            made.check(dtype, max_len, f"{D} {n} {nats} {dtype} {max_len}")


@pytest.mark.parametrize("D,n", [(64, 6000), (256, 3000)])
@pytest.mark.parametrize("nats,big", [(0, 2.0), (0, 20000.0), (12, 600.0), (12, 9000.0)])
def test_attention_large_group_beside_small_ones(D, n, nats, big):
    made = Tail(n, D, nats, big=big)
    for dtype in TYPES.values():
        for max_len in (1, n):
            made.check(dtype, max_len, f"{D} {n} {nats} {big} {dtype} {max_len}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("step", [-4.0, -0.5, 0.5, 4.0])
def test_attention_logits_that_fall_or_rise_with_every_page(D, step):
    """The weights' reference follows the pages down and up, by up to 160 nats; every
    eighth token has values over the whole of FP16's range."""
    n, H = 64 * 40 - 9, 1
    made = Made([n], H, D, seed=3, spread=0.0, v_scale=1.0)
    rng = np.random.default_rng(1)
    k = np.repeat(step * np.arange(n)[:, None] // 64, D, 1)[:, None].astype(np.float16)
    v = rng.standard_normal((n, H, D)).astype(np.float16)
    v[::8] = np.sign(v[::8]) * np.float16(65504)
    K4.append(made.data, made.summary, k, v, made.table[0, np.arange(n) // 64] * 64 + np.arange(n) % 64)
    cache = made.gpu()
    for dtype in TYPES.values():
        q = torch.ones(1, 2, D, dtype=dtype, device="cuda")
        for max_len in (1, n):
            lse = torch.empty(1, 2, device="cuda")
            out = cache.attention(q, ints(made.table), ints(made.lens), ints([0, 1]), 1, max_len, scale=1 / D, lse=lse)
            check_attention(out, lse, made, q, np.array([0, 1]), 1 / D, label=f"{D} {step} {dtype} {max_len}")
            check_held(out, made, q, np.array([0, 1]), 1 / D, f"{D} {step} {dtype} {max_len}")


# ---------------------------------------------------------- empty batches


@pytest.mark.parametrize("n_seqs", [0, 3])
def test_batches_without_rows(n_seqs):
    """Attention, selection and sparse attention of no rows return empty outputs."""
    made = Made([5, 70, 0], 2, 64)
    cache = made.gpu()
    q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    args = (ints(made.table[:n_seqs]), ints(made.lens[:n_seqs]), ints(np.zeros(n_seqs + 1)))
    assert cache.attention(q, *args, 0, 70).shape == q.shape
    sel = cache.select(q, *args, 4)
    assert sel.shape == (0, 2, 4)
    assert cache.attention(q, *args, 1 << 60, 1 << 60, sel=sel).shape == q.shape


# ---------------------------------------------------- memory and streams


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_on_another_stream_are_not_memory_in_use(handle):
    """The current stream still works on memory that it has given back: a call on
    another stream takes none of it for its output, its choice and its workspace."""
    made = Made([3000], 2, 64, seed=3)
    cache = made.gpu()
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(0)).half().cuda()
    args = (ints(made.table), ints(made.lens), ints([0, 1]))
    want, chosen = cache.attention(q, *args, 1, 3000), cache.select(q, *args, 5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20_000_000)
        used = [torch.full((n,), 2.0, device="cuda") for n in (16, 64, 1024, 4096, 65536)]
        held = [(t.data_ptr(), 4 * t.numel()) for t in used]
        sums = [t.sum() for t in used]
        del used
        out = cache.attention(q, *args, 1, 3000, stream=stream)
        sel = cache.select(q, *args, 5, stream=stream)
        for t in (out, sel):
            assert all(t.data_ptr() >= p + n or t.data_ptr() + t.numel() * t.element_size() <= p for p, n in held)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(sel, chosen)
        assert [float(s) for s in sums] == [32.0, 128.0, 2048.0, 8192.0, 131072.0]


@pytest.mark.parametrize("n_runs", [0, 5, 3000])
def test_plan_of_no_sequences(n_runs):
    """Fixed buffers of a step that has no sequences left: the last step's pages and
    runs are not taken again."""
    none, runs, taken = ints(np.zeros(0)), ints(np.full((n_runs, 2), 7)), ints([7])
    for cu in (none[:0].new_zeros(1), ints([0])):
        B.wq_kv4_plan(none, cu, ints(np.zeros((0, 4))), ints([3, 4]), none, none, runs, taken)
        assert int(taken) == 0 and (runs == ints([-1, 0])).all()


def test_plan_stays_in_bounds_for_any_rows():
    """cu_rows that fall, repeat and lie far outside the rows, over the longest
    lengths: every slot is of a page that the call was given, or none."""
    far = -(1 << 31)
    for cu, lens in (([far, 100, 200], [1 << 30, 5]), ([-(1 << 30) - 7, 100, 200], [1 << 30, 5]),
                     ([0, (1 << 31) - 1, 200], [70, 1 << 30]), ([5, far, (1 << 31) - 1], [70, 70])):
        slots, runs, taken = ints(np.zeros(300)), ints(np.zeros((8, 2))), ints([0])
        B.wq_kv4_plan(ints(lens), ints(cu), ints(np.full((2, 3), 50)), ints([60, 61]), ints([0, 0]), slots, runs, taken)
        assert set(np.unique(host(slots) // 64)) <= {-1, 50, 60, 61}, cu


def test_plan_stays_in_bounds_where_the_pages_overflow():
    """8192 sequences that claim all of 2^24 rows each: their pages pass 2^31."""
    n, T = 8192, 1 << 24
    cu = (np.arange(n + 1, dtype=np.int64) * T + (1 << 31)) % (1 << 32) - (1 << 31)
    slots, runs = ints(np.zeros(T)), ints(np.zeros((B.wq_kv4_max_runs(n, T), 2)))
    B.wq_kv4_plan(ints(np.ones(n)), ints(cu), ints(np.full((n, 2), 50)), ints([60, 61]), ints(np.zeros(n)), slots, runs,
                  ints([0]))
    assert set(torch.unique(slots.div(64, rounding_mode="floor")).tolist()) <= {-1, 50, 60, 61}


@pytest.mark.parametrize("D", [64, 128])
def test_attention_stays_in_bounds_for_any_rows(D):
    """cu_rows and lengths at the ends of int32: nothing outside the given rows is
    written, and sequences that are in order keep their results."""
    made = Made([100, 50, 200], 2, D, seed=2)
    cache = made.gpu()
    q = torch.randn(70, 4, D, generator=torch.Generator().manual_seed(3)).half().cuda()
    low, high = -(1 << 31), (1 << 31) - 1
    room = torch.empty(90, 4, D, dtype=torch.float16, device="cuda")
    table = ints(made.table)
    for max_rows in (1, 70):
        want = cache.attention(q, table, ints(made.lens), ints([0, 6, 6, 70]), max_rows, 200)
        for cu in ([0, 6, low, 70], [0, 6, high, low], [low, 6, low, high], [high, high, low, low], [0, 6, 70, low]):
            for lens in ([100, 50, 200], [100, low, high]):
                room.fill_(5.0)
                cache.attention(q, table, ints(lens), ints(cu), max_rows, 200, out=room[10:80])
                assert (room[:10] == 5).all() and (room[80:] == 5).all(), (cu, lens)
                if cu[:2] == [0, 6] and cu[2] >= 70:            # no sequence shares rows 0 .. 5
                    assert torch.equal(room[10:16], want[:6]), (cu, lens)
                sel = cache.select(q, table, ints(lens), ints(cu), 2)
                assert int(sel.min()) >= -1 and int(sel.max()) < made.table.shape[1]
                room.fill_(5.0)
                cache.attention(q, table, ints(lens), ints(cu), max_rows, 200, sel=sel, out=room[10:80])
                assert (room[:10] == 5).all() and (room[80:] == 5).all(), (cu, lens)


# ------------------------------------------------- bounds of any query


def choose(made, q, n_sel, label):
    cu = [0, len(q)]
    sel = made.gpu().select(q, ints(made.table), ints(made.lens), ints(cu), n_sel)
    assert np.array_equal(host(sel), K4.select(made.summary, f32(q), made.table, made.lens, cu, n_sel)), label


def test_select_keeps_the_last_page_beside_bounds_past_float32():
    made = Made([64 * 30 + 1], 1, 128, seed=4, spread=3.0)
    for size in (1e37, 3e38):
        q = (size * torch.sign(torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(5)))).to(torch.bfloat16)
        for n in (2, 5, 20):
            choose(made, q.cuda(), n, f"{size} {n}")


@pytest.mark.parametrize("heads", [2, 6, 20])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_select_with_queries_that_are_not_finite(dtype, heads):
    """A head whose query holds an infinity or NaN does not decide for its group,
    also where a channel's minimum and maximum are equal, 0 or of two signs."""
    made = Made([64 * 40 + 9], 2, 64, seed=4)
    made.summary[made.table[0, 3], :, :, 5] = 0
    made.summary[made.table[0, 4], :, 0, 5] = made.summary[made.table[0, 4], :, 1, 5]
    q = torch.randn(2, heads, 64, generator=torch.Generator().manual_seed(5)).to(TYPES[dtype])
    for bad in (float("inf"), -float("inf"), float("nan")):
        one, two, whole = q.clone(), q.clone(), q.clone()
        one[1, heads // 2, 5] = bad
        two[0, 0, 5], two[0, heads - 1, 60] = bad, -bad
        whole[0, :, 7] = bad
        for n in (2, 7):
            for x in (one, two, whole):
                choose(made, x.cuda(), n, f"{dtype} {heads} {bad} {n}")


def test_strides_of_single_rows_and_heads_do_not_count():
    """One row of a buffer whose rows are no multiple of 8 long, one head likewise."""
    D = 64
    made = Made([70], 1, D, seed=6)
    cache = made.gpu()
    wide = torch.randn(1, 5 * D + 3, generator=torch.Generator().manual_seed(3)).half().cuda()
    q = wide[:, :4 * D].view(1, 4, D)
    out = cache.attention(q, ints(made.table), ints(made.lens), ints([0, 1]), 1, 70)
    check_attention(out, None, made, q, np.array([0, 1]), D ** -0.5, label="one row")
    sel = cache.select(q, ints(made.table), ints(made.lens), ints([0, 1]), 2)
    assert np.array_equal(host(sel), K4.select(made.summary, f32(q), made.table, made.lens, [0, 1], 2))
    k = torch.randn(2, 80, D, generator=torch.Generator().manual_seed(4)).half().cuda()
    k, v = (x.as_strided((80, 1, D), (D, 3, 1)) for x in k)
    slots = np.arange(80)[:50] + 64 * made.table[0, 0]
    cache.append(k[:50], v[:50], ints(slots), ints([[0, 50]]))
    K4.append(made.data, made.summary, f32(k[:50]), f32(v[:50]), slots)
    assert np.array_equal(made.d.cpu().numpy(), made.data)


# ------------------------------------------- splits, turns and long tables


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [63, 300, 1000, 4000])
def test_attention_window_over_several_splits(D, window):
    """Windows that begin inside a late page of a long cache, whole call and one workgroup."""
    made = Made([5000, 1700], 1, D, seed=13)
    cache = made.gpu()
    for dtype in TYPES.values():
        for rows in ([1, 1], [3, 40]):
            for max_len in (1, 5000, 1 << 20):
                attend(made, cache, rows, 2, dtype, window=window, max_len=max_len,
                       label=f"{D} window {window} {rows} {max_len}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 900])
def test_attention_two_column_tiles_over_several_splits(D, window):
    """Rows enough for two column tiles a wave, over splits, and over so many pages a
    wave that it folds its sums on the way."""
    made = Made([2611, 700], 1, D, seed=14, v_scale=2.0)
    cache = made.gpu()
    for dtype in TYPES.values():
        for max_len in (1, 2611):
            attend(made, cache, [40, 33], 2, dtype, window=window, max_len=max_len,
                   label=f"{D} two tiles {window} {max_len}")


class Pages:
    """Summaries of many pages alone, for selection."""

    def __init__(self, lens, H, D, seed=0):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens)
        need = -(-self.lens // 64)
        self.table = np.full((len(lens), int(need.max()) + 3), -1)
        order = rng.permutation(int(need.sum()) + 2)
        for b, n in enumerate(need):
            self.table[b, :n] = order[need[:b].sum():][:n]
        centre = rng.standard_normal((len(order), H, D))
        half = np.abs(rng.standard_normal((len(order), H, D)))
        self.summary = np.stack([centre - half, centre + half], 2).astype(np.float16)
        self.cache = B.KV4Cache(torch.zeros(len(order), H, 80 * D, dtype=torch.uint8, device="cuda"),
                                torch.from_numpy(self.summary).cuda())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,rows,heads,n_sel", [([64 * 1100 - 5, 64 * 500], [12, 8], 2, 33), ([64 * 600], [16], 24, 9),
                                                   ([64 * 9001, 70], [1, 1], 2, 40)])
def test_select_over_many_pages(D, dtype, lens, rows, heads, n_sel):
    """Several turns of a wave, more than 8 heads a group, and a table whose keys do
    not fit the workgroup's memory."""
    H = 1 if len(lens) == 2 and lens[1] == 70 else 2
    made = Pages(lens, H, D, seed=D + heads)
    cu = np.concatenate([[0], np.cumsum(rows)])
    q = torch.randn(int(cu[-1]), heads, D, generator=torch.Generator().manual_seed(2)).to(TYPES[dtype]).cuda()
    sel = made.cache.select(q, ints(made.table), ints(made.lens), ints(cu), n_sel)
    assert np.array_equal(host(sel), K4.select(made.summary, f32(q), made.table, made.lens, cu, n_sel))
