"""4-bit key/value cache, on the CPU: the oracle's layout and format against
what the header says of them, and the entry points' refusals."""

import ctypes

import numpy as np
import pytest

import bit_weight_only_gemv_amd as B
from bit_weight_only_gemv_amd import _lib as L
from oracle import kv4_oracle as K4


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_holds_every_bit_once(D):
    P = K4._places(D)
    seen = np.zeros(80 * D, np.int64)          # half bytes used
    for name in ("k", "v"):
        byte, shift = P[name]
        assert set(np.unique(shift)) == {0, 4}
        np.add.at(seen, byte.reshape(-1), 1)
        assert len(set(zip(byte.reshape(-1), shift.reshape(-1)))) == 64 * D
    for name in ("ks", "kz", "vs", "vz"):
        for o in (0, 1):
            np.add.at(seen, P[name].reshape(-1) + o, 2)
    assert (seen == 2).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tokens_read_back_as_quantized(D):
    rng = np.random.default_rng(D)
    k, v = rng.standard_normal((2, 64, D)).astype(np.float16)
    page = rng.integers(0, 256, 80 * D, dtype=np.uint8)
    for t in rng.permutation(64):
        K4.write_token(page, t, k[t], v[t])
    kr, vr, size = K4.read_page(page, D)
    assert np.array_equal(kr, K4.dequantize(*K4.quantize(k)))
    assert np.array_equal(vr, K4.dequantize(*K4.quantize(v)))
    assert (size >= np.abs(kr) * (1 - 1e-12)).all()


def test_quantization_error_and_edges():
    rng = np.random.default_rng(3)
    w = (rng.standard_normal((50, 32)) * 10.0 ** rng.integers(-3, 4, (50, 1))).astype(np.float32)
    q, s, z = K4.quantize(w)
    err = np.abs(K4.dequantize(q, s, z) - w)
    # half a step, and where S or Z was rounded, what the ends lose by it: half
    # an FP16 step of Z and 15 half steps of S (2^-11 relative, 2^-25 absolute)
    span = w.max(-1) - w.min(-1)
    lim = 0.5 * s.astype(float)[:, 0] + 2.0 ** -11 * (np.abs(w.min(-1)) + span) + 16 * 2.0 ** -25
    assert (err <= lim[:, None] * (1 + 1e-6)).all()
    for row in ([0.0] * 32, [7.5] * 32, [-65504.0] * 16 + [65504.0] * 16):
        q, s, z = K4.quantize(np.array(row, np.float32))
        assert np.allclose(K4.dequantize(q, s, z), row, rtol=2.0 ** -10)
    q, s, z = K4.quantize(np.array([np.nan, np.inf, -np.inf] + [1.0] * 29, np.float32))
    assert np.isfinite(K4.dequantize(q, s, z)).all()


# ------------------------------------------------------------- refusals


P = 4096        # a 16-byte aligned address; refused calls never read it


def cache(data=P, summary=P, pages=10, heads=2, dim=128):
    return L.Kv4Cache(data, summary, pages, heads, dim)


def rows(**kw):
    a = dict(block_table=P, lens=P, cu_rows=P, table_width=4, n_seqs=2, n_rows=2, n_heads=8, dtype=0,
             q=P, q_row_stride=1024, q_head_stride=128)
    a.update(kw)
    return L.Kv4Rows(**a)


def ref(s):
    return ctypes.addressof(s) if s is not None else None


def attend(c=None, a=None, max_rows=1, max_len=64, window=0, sel=None, n_sel=0, out=P, lse=None,
           ws=P, ws_bytes=1 << 40):
    c, a = c or cache(), a or rows()
    return L.load().wq_kv4_attention(ref(c), ref(a), max_rows, max_len, 0.1, window, sel, n_sel, out,
                                     lse, ws, ws_bytes, None)


def choose(c=None, a=None, n_sel=4, sel=P, ws=P, ws_bytes=1 << 40):
    c, a = c or cache(), a or rows()
    return L.load().wq_kv4_select(ref(c), ref(a), n_sel, sel, ws, ws_bytes, None)


def append(c=None, dtype=0, k=P, kr=256, kh=128, v=P, vr=256, vh=128, n=2, slots=P, runs=P, n_runs=2):
    c = c or cache()
    return L.load().wq_kv4_append(ref(c), dtype, k, kr, kh, v, vr, vh, n, slots, runs, n_runs, None)


def plan(lens=P, cu=P, B_=2, T=4, table=P, width=4, free=P, n_free=4, new=P, slots=P, runs=P, n_runs=4,
         taken=P):
    return L.load().wq_kv4_plan(lens, cu, B_, T, table, width, free, n_free, new, slots, runs, n_runs,
                                taken, None)


BAD_CACHE = [(dict(data=None), -1), (dict(data=P + 8), -1), (dict(summary=P + 2), -1), (dict(pages=0), -1),
             (dict(pages=1 << 40), -1), (dict(heads=0), -1), (dict(dim=96), -2), (dict(dim=0), -2),
             (dict(dim=-128), -2)]
BAD_ROWS = [(dict(block_table=None), -1), (dict(lens=None), -1), (dict(lens=P + 2), -1), (dict(block_table=P + 1), -1), (dict(cu_rows=None), -1), (dict(q=None), -1),
            (dict(q=P + 2), -1), (dict(table_width=0), -1), (dict(n_seqs=-1), -1), (dict(n_rows=-1), -1),
            (dict(n_heads=7), -1), (dict(n_heads=0), -1), (dict(dtype=2), -2), (dict(q_row_stride=1020), -1),
            (dict(q_head_stride=4), -1), (dict(q_row_stride=-1024), -1)]


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_refuses_bad_caches(bad, status):
    c = cache(**bad)
    for call in (attend, append, choose):
        assert call(c) == status
        assert L.load().wq_last_error()


@pytest.mark.parametrize("bad,status", BAD_ROWS)
def test_refuses_bad_rows(bad, status):
    a = rows(**bad)
    for call in (attend, choose):
        assert call(a=a) == status
        assert L.load().wq_last_error()


@pytest.mark.parametrize("call,bad", [
    (attend, dict(max_rows=-1)), (attend, dict(max_len=-1)), (attend, dict(window=-1)),
    (attend, dict(n_sel=-1)), (attend, dict(out=None)), (attend, dict(out=P + 4)),
    (attend, dict(lse=P + 2)), (attend, dict(sel=P + 2, n_sel=4)), (attend, dict(ws=P + 4)),
    (choose, dict(n_sel=1)), (choose, dict(n_sel=0)), (choose, dict(sel=None)), (choose, dict(ws=None)),
    (choose, dict(ws_bytes=8)), (choose, dict(c=cache(summary=None))), (choose, dict(ws=P + 4)),
    (append, dict(k=None)), (append, dict(v=None)), (append, dict(k=P + 2)), (append, dict(v=P + 8)),
    (append, dict(kr=250)), (append, dict(vh=4)), (append, dict(kr=-256)), (append, dict(slots=None)),
    (append, dict(runs=None)), (append, dict(n=-1)), (append, dict(n_runs=-1)), (append, dict(runs=P + 4)),
    (append, dict(n_runs=1 << 40)),
    (plan, dict(lens=None)), (plan, dict(cu=None)), (plan, dict(table=None)), (plan, dict(new=None)),
    (plan, dict(slots=None)), (plan, dict(runs=None)), (plan, dict(taken=None)), (plan, dict(free=None)),
    (plan, dict(n_runs=3)), (plan, dict(width=0)), (plan, dict(B_=-1)), (plan, dict(T=-1)),
    (plan, dict(n_free=-1)), (plan, dict(lens=P + 2)), (plan, dict(free=P + 1)), (plan, dict(runs=P + 4)),
])
def test_refuses_bad_arguments(call, bad):
    assert call(**bad) == L.WQ_ERR_INVALID_ARG
    assert L.load().wq_last_error()


def test_refuses_what_is_not_supported():
    assert append(dtype=3) == L.WQ_ERR_UNSUPPORTED
    assert plan(B_=L.WQ_KV4_MAX_SEQS + 1, n_runs=1 << 20) == L.WQ_ERR_UNSUPPORTED
    assert L.load().wq_kv4_append(None, 0, P, 8, 8, P, 8, 8, 1, P, P, 1, None) == L.WQ_ERR_INVALID_ARG
    assert L.load().wq_kv4_attention(ref(cache()), None, 1, 1, 1.0, 0, None, 0, P, None, P, 0, None) == -1


def test_empty_calls_do_nothing():
    assert attend(a=rows(n_rows=0)) == 0 and attend(a=rows(n_seqs=0)) == 0
    assert choose(a=rows(n_rows=0)) == 0
    assert append(n=0) == 0 and append(n_runs=0) == 0
    assert plan(B_=0) == 0


def test_sizes():
    assert B.wq_kv4_max_runs(0, 0) == 0
    assert B.wq_kv4_max_runs(64, 64) == 64
    assert B.wq_kv4_max_runs(3, 1000) == 21
    with pytest.raises(B.WQError):
        B.wq_kv4_max_runs(-1, 5)
    assert L.load().wq_kv4_select_workspace(3, 2, 5) == 128
    assert L.load().wq_kv4_select_workspace(-1, 2, 5) < 0
    assert L.load().wq_kv4_attention_workspace(ref(cache(dim=96)), ref(rows()), 1, 64, 0) < 0


def test_runs_never_exceed_their_bound():
    rng = np.random.default_rng(5)
    for _ in range(300):
        n = int(rng.integers(1, 9))
        lens = rng.integers(0, 200, n)
        new = rng.integers(0, int(rng.integers(1, 200)), n)
        cu = np.concatenate([[0], np.cumsum(new)])
        table = np.zeros((n, 10), np.int64)
        _, _, slots, runs, _ = K4.plan(lens, cu, table, np.arange(100))
        assert len(runs) == B.wq_kv4_max_runs(n, int(cu[-1]))
        assert runs[:, 1].sum() == cu[-1]


def test_wrapper_checks():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        B.KV4Cache(torch.zeros(2, 2, 100, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.KV4Cache(torch.zeros(2, 2, 80 * 64, dtype=torch.uint8))     # not on the GPU
    with pytest.raises(ValueError):
        B.KV4Cache(torch.zeros(2, 2, 80 * 64, dtype=torch.uint8), torch.zeros(2, 2, 2, 32, dtype=torch.float16))


def space(c=None, a=None, max_rows=1, max_len=64, n_sel=0):
    c, a = c or cache(), a or rows()
    return L.load().wq_kv4_attention_workspace(ref(c), ref(a), max_rows, max_len, n_sel)


@pytest.mark.parametrize("n_rows,n_seqs,n_sel", [(0, 0, 0), (0, 2, 0), (0, 2, 4), (2, 0, 0), (2, 0, 4)])
def test_empty_batches_need_no_workspace(n_rows, n_seqs, n_sel):
    assert space(a=rows(n_rows=n_rows, n_seqs=n_seqs), n_sel=n_sel) == 0


def test_an_empty_batch_may_have_an_empty_list():
    assert attend(a=rows(n_rows=0), sel=None, n_sel=4) == 0
    assert attend(sel=None, n_sel=4) == attend(sel=P, n_sel=0) == L.WQ_ERR_INVALID_ARG


@pytest.mark.parametrize("n_heads", [8, 32, 64])
@pytest.mark.parametrize("big", [1 << 31, 1 << 58, 1 << 62, (1 << 63) - 1])
def test_hints_beyond_the_call_count_as_its_size(n_heads, big):
    """Rows and lengths that the call cannot have: n_rows and 64 table_width of them."""
    a = rows(n_rows=50, n_heads=n_heads, table_width=900)
    assert space(a=a, max_rows=big, max_len=big) == space(a=a, max_rows=50, max_len=64 * 900) > 0
    assert space(a=a, max_rows=1, max_len=big) == space(a=a, max_rows=1, max_len=64 * 900) > 0


@pytest.mark.parametrize("handle", [False, True])
def test_memory_made_for_a_stream_comes_from_that_stream(monkeypatch, handle):
    """A block that the current stream has just given back may still be in use there,
    and a call on another stream does not wait for it: what such a call writes has
    to be memory of its own stream.  What it returns is also held for the current
    one, where the caller uses and drops it; its workspace is not."""
    import contextlib

    torch = pytest.importorskip("torch")
    from bit_weight_only_gemv_amd import kv4

    class Stream:
        def __init__(self, handle=7, device=None):
            self.cuda_stream = handle

    current, made = Stream(1), []
    now = [current]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    class Tensor:
        def __init__(self, *a, **kw):
            self.of, self.held = now[-1].cuda_stream, []
            made.append(self)

        def numel(self):
            return 4

        def record_stream(self, s):
            self.held.append(s.cuda_stream)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", Tensor)
    t = kv4._new((4,), torch.uint8, "cuda", 9 if handle else Stream(9))
    assert t.of == 9 and t.held == [1]
    t = kv4._new((4,), torch.uint8, "cuda", None)
    assert t.of == 1 and t.held == []
    t = kv4._workspace(4, "cuda", 9 if handle else Stream(9))
    assert t.of == 9 and t.held == []
    assert now == [current] and len(made) == 3


def test_wrappers_refuse_rows_of_no_sequences():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    none, cu, table = torch.zeros(0, **i32), torch.zeros(1, **i32), torch.zeros(0, 4, **i32)
    with pytest.raises(ValueError, match="no sequences"):
        B.wq_kv4_plan(none, cu, table, none, none, torch.zeros(3, **i32), torch.zeros(3, 2, **i32), cu)
    c = object.__new__(B.KV4Cache)
    c.n_kv_heads, c.head_dim = 2, 64
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="no sequences"):
        c.select(q, table, none, cu, 4)
    with pytest.raises(ValueError, match="no sequences"):
        c.attention(q, table, none, cu, 1, 64)


def test_plan_of_no_sequences_needs_no_tables_but_taken():
    none = dict(B_=0, T=0, lens=None, cu=None, table=None, new=None, slots=None, free=None, n_free=0)
    assert plan(**none, taken=None) == L.WQ_ERR_INVALID_ARG
    assert plan(**none, n_runs=4, runs=None) == L.WQ_ERR_INVALID_ARG


def test_attention_refuses_a_list_without_places():
    """Its pointer is NULL, which would mean all tokens."""
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    c = object.__new__(B.KV4Cache)
    c.n_kv_heads, c.head_dim = 2, 64
    q = torch.zeros(1, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="sel"):
        c.attention(q, torch.zeros(1, 4, **i32), torch.zeros(1, **i32), torch.zeros(2, **i32), 1, 64,
                    sel=torch.zeros(1, 2, 0, **i32))


@pytest.mark.parametrize("n_rows,heads,width", [(1 << 24, 65535, 1 << 24), (1 << 24, 128, 1)])
def test_select_workspace_refuses_what_select_does(n_rows, heads, width):
    """Sizes whose bytes would wrap, or that the call itself does not take."""
    assert L.load().wq_kv4_select_workspace(n_rows, heads, width) == L.WQ_ERR_UNSUPPORTED
    assert L.load().wq_last_error()
