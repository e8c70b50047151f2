"""8-bit key/value cache, eviction, norm and rotation: the oracle's own properties, and what
the library and its wrappers refuse (no GPU: refused and empty calls launch nothing)."""

import ctypes

import numpy as np
import pytest

import bit_weight_only_gemv_amd as B
from bit_weight_only_gemv_amd import _lib as L
from oracle import kv8_oracle as K8

# ------------------------------------------------------------- the format


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_is_a_bijection(D):
    k, v = K8.places(D)
    assert np.array_equal(np.sort(np.concatenate([k.ravel(), v.ravel()])), np.arange(128 * D))


def test_exponents():
    assert K8.exponent(0.0) == K8.exponent(127.49 * 2.0 ** -24) == -24
    assert K8.exponent(127.5 * 2.0 ** -24) == -23
    assert K8.exponent(127.0) == 0 and K8.exponent(127.5) == 1 and K8.exponent(63.75) == 0
    assert K8.exponent(63.74) == -1 and K8.exponent(65504.0) == 10


@pytest.mark.parametrize("steps", [(64,), (1,) * 64, (5, 11, 1, 30, 17), (16, 16, 32)])
def test_appended_values_are_within_their_steps(steps):
    """Half a step of the block's exponent, and another for every time it rose."""
    D, H = 64, 2
    rng = np.random.default_rng(len(steps))
    k, v = (rng.standard_normal((2, 64, H, D)) * np.exp(0.5 * rng.standard_normal((2, 64, 1, 1)))).astype(np.float16)
    data, exps = np.zeros((1, H, 128 * D), np.uint8), np.zeros((1, H, 8), np.int8)
    at, rises = 0, np.zeros((H, 8))
    for n in steps:
        before = exps[0].astype(int)
        K8.append(data, exps, k[at:at + n], v[at:at + n], np.arange(at, at + n), [[0, n]])
        held = np.repeat(np.arange(4) * 16 < at, 1)
        rises += (exps[0] > before) & np.tile(held, 2)[None]
        at += n
    for h in range(H):
        for got, want, first in zip(K8.read_page(data[0, h], exps[0, h], D), (k[:, h], v[:, h]), (0, 4)):
            step = np.repeat(2.0 ** exps[0, h, first:first + 4].astype(float), 16)[:, None]
            lim = step * (0.5 + 0.5 * np.repeat(rises[h, first:first + 4], 16)[:, None])
            assert (np.abs(got - want) <= lim).all()


def test_whole_blocks_do_not_depend_on_the_calls():
    D, rng = 64, np.random.default_rng(0)
    k, v = rng.standard_normal((2, 64, 1, D)).astype(np.float32)
    a = np.zeros((1, 1, 128 * D), np.uint8), np.zeros((1, 1, 8), np.int8)
    b = np.zeros((1, 1, 128 * D), np.uint8), np.zeros((1, 1, 8), np.int8)
    K8.append(*a, k, v, np.arange(64), [[0, 64]])
    for t in range(0, 64, 16):
        K8.append(*b, k[t:t + 16], v[t:t + 16], np.arange(t, t + 16), [[0, 16]])
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_rotation_keeps_lengths_and_depends_on_distance():
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(32) / 32)
    q, k = rng.standard_normal((2, 1, 1, 64))
    for n in (False, True):
        at = lambda x, p: K8.norm_rope(x, None, [p], f, None, n)[0][0, 0]  # noqa: E731
        assert np.allclose(at(q, 5) @ at(k, 2), at(q, 105) @ at(k, 102))
        assert np.allclose(np.linalg.norm(at(q, 77)), np.linalg.norm(q))


# --------------------------------------------------------------- refusals

P = 4096        # a 16-byte aligned address; refused calls never read it


def cache(data=P, exps=P, pages=10, heads=2, dim=128):
    return L.Kv8Cache(data, exps, pages, heads, dim)


def rows(**kw):
    a = dict(block_table=P, lens=P, cu_rows=P, table_width=4, n_seqs=2, n_rows=2, n_heads=8, dtype=0,
             q=P, q_row_stride=1024, q_head_stride=128)
    a.update(kw)
    return L.Kv4Rows(**a)


def ref(s):
    return ctypes.addressof(s) if s is not None else None


def attend(c=None, a=None, max_rows=1, max_len=64, window=0, out=P, lse=None, ws=P, ws_bytes=1 << 40):
    c, a = c or cache(), a or rows()
    return L.load().wq_kv8_attention(ref(c), ref(a), max_rows, max_len, 0.1, window, out, lse, ws, ws_bytes, None)


def append(c=None, dtype=0, k=P, kr=256, kh=128, v=P, vr=256, vh=128, n=2, slots=P, runs=P, n_runs=2):
    c = c or cache()
    return L.load().wq_kv8_append(ref(c), dtype, k, kr, kh, v, vr, vh, n, slots, runs, n_runs, None)


def accumulate(c=None, a=None, max_rows=1, max_len=64, lse=P, window=0, held=P, mass=P, tokens=256, ws=P,
               ws_bytes=1 << 40):
    c, a = c or cache(), a or rows()
    return L.load().wq_kv8_accumulate(ref(c), ref(a), max_rows, max_len, lse, 0.1, window, held, mass, tokens,
                                      ws, ws_bytes, None)


def evict(c=None, mass=P, tokens=256, table=P, width=4, lens=P, B_=2, keep=100, recent=10, free=P, n_free=4,
          new_table=2 * P, new_lens=2 * P, new_mass=2 * P, new_tokens=100, taken=P, kept=P):
    c = c or cache()
    return L.load().wq_kv8_evict(ref(c), mass, tokens, table, width, lens, B_, keep, recent, free, n_free, new_table,
                                 new_lens, new_mass, new_tokens, taken, kept, None)


def heads(**kw):
    a = dict(x=P, out=2 * P, weight=P, n_heads=4, row_stride=1024, head_stride=128, out_row_stride=512, out_head_stride=128)
    a.update(kw)
    return L.Heads(**a)


def rope(q=None, k=None, dtype=0, T=3, D=128, eps=1e-6, pos=P, freq=P, n=64, nb=0):
    q, k = q or heads(), k or heads()
    return L.load().wq_qk_norm_rope(dtype, ref(q), ref(k), T, D, eps, pos, freq, n, nb, None)


BAD_CACHE = [(dict(data=None), -1), (dict(data=P + 8), -1), (dict(exps=None), -1), (dict(exps=P + 4), -1),
             (dict(pages=0), -1), (dict(pages=1 << 40), -1), (dict(heads=0), -1), (dict(dim=96), -2), (dict(dim=0), -2)]
BAD_ROWS = [(dict(block_table=None), -1), (dict(lens=P + 2), -1), (dict(cu_rows=None), -1), (dict(q=None), -1),
            (dict(q=P + 2), -1), (dict(table_width=0), -1), (dict(n_seqs=-1), -1), (dict(n_rows=-1), -1),
            (dict(n_heads=7), -1), (dict(dtype=2), -2), (dict(q_row_stride=1020), -1), (dict(q_row_stride=-1024), -1)]


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_refuses_bad_caches(bad, status):
    c = cache(**bad)
    for call in (attend, append, accumulate, evict):
        assert call(c) == status
        assert L.load().wq_last_error()
    assert L.load().wq_kv8_attention_workspace(ref(c), ref(rows()), 1, 64) == status
    assert L.load().wq_kv8_accumulate_workspace(ref(c), ref(rows()), 1, 64) == status


@pytest.mark.parametrize("bad,status", BAD_ROWS)
def test_refuses_bad_rows(bad, status):
    a = rows(**bad)
    for call in (attend, accumulate):
        assert call(a=a) == status
        assert L.load().wq_last_error()


@pytest.mark.parametrize("call,bad", [
    (attend, dict(max_rows=-1)), (attend, dict(max_len=-1)), (attend, dict(window=-1)), (attend, dict(out=None)),
    (attend, dict(out=P + 4)), (attend, dict(lse=P + 2)), (attend, dict(ws=P + 4)),
    (append, dict(k=None)), (append, dict(v=None)), (append, dict(k=P + 2)), (append, dict(v=P + 8)),
    (append, dict(kr=250)), (append, dict(vh=4)), (append, dict(kr=-256)), (append, dict(slots=None)),
    (append, dict(runs=None)), (append, dict(n=-1)), (append, dict(n_runs=-1)), (append, dict(runs=P + 4)),
    (append, dict(n_runs=1 << 40)), (append, dict(n_runs=1 << 62)),
    (accumulate, dict(max_rows=-1)), (accumulate, dict(max_len=-1)), (accumulate, dict(window=-1)),
    (accumulate, dict(lse=None)), (accumulate, dict(lse=P + 2)), (accumulate, dict(held=None)),
    (accumulate, dict(held=P + 1)), (accumulate, dict(mass=None)), (accumulate, dict(mass=P + 2)),
    (accumulate, dict(tokens=0)),
    (evict, dict(mass=None)), (evict, dict(mass=P + 2)), (evict, dict(tokens=0)), (evict, dict(table=None)),
    (evict, dict(width=0)), (evict, dict(width=1)), (evict, dict(lens=None)), (evict, dict(B_=-1)), (evict, dict(keep=0)),
    (evict, dict(keep=257, new_tokens=300)), (evict, dict(recent=-1)), (evict, dict(recent=101)),
    (evict, dict(free=None)), (evict, dict(n_free=-1)), (evict, dict(new_table=None)), (evict, dict(new_table=P)),
    (evict, dict(new_lens=None)), (evict, dict(new_lens=P)), (evict, dict(new_mass=None)), (evict, dict(new_mass=P)),
    (evict, dict(new_tokens=99)), (evict, dict(taken=None)), (evict, dict(taken=P + 2)), (evict, dict(kept=None)),
    (evict, dict(kept=P + 2)), (evict, dict(keep=1 << 40, new_tokens=1 << 41)),
    (rope, dict(T=-1)), (rope, dict(T=1 << 30)), (rope, dict(n=-4)), (rope, dict(n=6)), (rope, dict(n=68)),
    (rope, dict(pos=None)), (rope, dict(pos=P + 2)), (rope, dict(freq=None)), (rope, dict(freq=P + 4)),
    (rope, dict(eps=float("nan"))), (rope, dict(q=heads(x=None))), (rope, dict(k=heads(out=None))),
    (rope, dict(q=heads(x=P + 2))), (rope, dict(q=heads(out=P + 8))), (rope, dict(k=heads(weight=P + 4))),
    (rope, dict(q=heads(row_stride=1020))), (rope, dict(q=heads(out_head_stride=4))), (rope, dict(k=heads(head_stride=-128))),
    (rope, dict(q=heads(out_row_stride=0))), (rope, dict(k=heads(out_head_stride=0))), (rope, dict(k=heads(out_head_stride=64))),
    (rope, dict(q=heads(n_heads=-1))), (rope, dict(q=heads(n_heads=1 << 20))), (rope, dict(q=heads(out=P))),
])
def test_refuses_bad_arguments(call, bad):
    assert call(**bad) == L.WQ_ERR_INVALID_ARG
    assert L.load().wq_last_error()


def test_refuses_what_is_not_supported():
    assert append(dtype=3) == rope(dtype=2) == rope(D=96) == rope(D=0, n=0) == L.WQ_ERR_UNSUPPORTED
    assert evict(B_=L.WQ_KV4_MAX_SEQS + 1) == L.WQ_ERR_UNSUPPORTED
    big = rows(n_rows=1 << 24, n_heads=65534)
    assert attend(a=big, ws_bytes=1 << 62) == accumulate(a=big, ws_bytes=1 << 62) == L.WQ_ERR_UNSUPPORTED
    assert L.load().wq_qk_norm_rope(0, None, ref(heads()), 1, 64, 0.0, P, P, 4, 0, None) == L.WQ_ERR_INVALID_ARG


def test_empty_calls_do_nothing():
    assert attend(a=rows(n_rows=0)) == attend(a=rows(n_seqs=0)) == 0
    assert accumulate(a=rows(n_rows=0)) == accumulate(a=rows(n_seqs=0)) == 0
    assert append(n=0) == append(n_runs=0) == 0
    assert rope(T=0) == 0
    assert rope(q=heads(n_heads=0, x=None, out=None, weight=None), k=heads(n_heads=0, x=None, out=None, weight=None)) == 0


def test_evict_of_no_sequences_needs_no_tables_but_taken():
    none = dict(B_=0, mass=None, table=None, lens=None, free=None, n_free=0, new_table=None, new_lens=None, new_mass=None, kept=None)
    assert evict(**none, taken=None) == evict(**none, taken=P + 2) == L.WQ_ERR_INVALID_ARG


def test_workspaces_are_needed_where_they_are_asked_for():
    """Many rows: scaled queries; long sequences: parts of splits.  Sizes grow with both."""
    many, few = rows(n_rows=50, n_heads=32, table_width=900), rows()
    need = L.load().wq_kv8_accumulate_workspace(ref(cache()), ref(many), 50, 64)
    assert need >= 50 * 32 * 128 * 2 and L.load().wq_kv8_accumulate_workspace(ref(cache()), ref(few), 1, 64) == 0
    parts = L.load().wq_kv8_attention_workspace(ref(cache()), ref(many), 1, 64 * 900)
    assert parts >= 50 * 32 * 128 * 4
    for bad in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=P + 8)):
        assert accumulate(a=many, max_rows=50, **bad) == L.WQ_ERR_INVALID_ARG
    for bad in (dict(ws=None), dict(ws_bytes=parts - 1), dict(ws=P + 8)):
        assert attend(a=many, max_len=64 * 900, **bad) == L.WQ_ERR_INVALID_ARG


@pytest.mark.parametrize("big", [1 << 31, 1 << 58, (1 << 63) - 1])
def test_hints_beyond_the_call_count_as_its_size(big):
    a = rows(n_rows=50, n_heads=32, table_width=900)
    for f in (L.load().wq_kv8_attention_workspace, L.load().wq_kv8_accumulate_workspace):
        space = lambda r, n: f(ref(cache()), ref(a), r, n)  # noqa: E731
        assert space(big, big) == space(50, 64 * 900) >= 0
        assert space(1, big) == space(1, 64 * 900) >= 0


def test_wrapper_checks():
    torch = pytest.importorskip("torch")
    u8, i8, i32 = (dict(dtype=t) for t in (torch.uint8, torch.int8, torch.int32))
    for data, exps in (((2, 2, 100), (2, 2, 8)), ((2, 2, 128 * 64), (2, 2, 4)), ((2, 2, 128 * 64), (2, 2, 8))):
        with pytest.raises(ValueError):                 # the last is not on the GPU
            B.KV8Cache(torch.zeros(*data, **u8), torch.zeros(*exps, **i8))
    c = object.__new__(B.KV8Cache)
    c.n_kv_heads, c.head_dim = 2, 64
    none, cu, table = torch.zeros(0, **i32), torch.zeros(1, **i32), torch.zeros(0, 4, **i32)
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="no sequences"):
        c.attention(q, table, none, cu, 1, 64)
    with pytest.raises(ValueError, match="no sequences"):
        c.accumulate(q, torch.zeros(3, 4), table, none, cu, none, torch.zeros(0, 2, 64), 1, 64)
    with pytest.raises(ValueError):
        c.append(q, q, torch.zeros(3, **i32), torch.zeros(3, 2, **i32))      # 4 heads, not 2
    with pytest.raises(ValueError):
        c.evict(torch.zeros(2, 64), torch.zeros(2, 1, **i32), torch.zeros(2, **i32), 5, 1, none, table, none,
                torch.zeros(2, 2, 5), cu)


def test_workspaces_of_another_device_are_refused(monkeypatch):
    """Before the library sees them: a launch would write there."""
    torch = pytest.importorskip("torch")

    class OnGpu:
        """What the wrappers ask of a contiguous tensor on GPU `at`."""
        is_cuda, device = True, "cuda"

        def __init__(self, shape, dtype, at=0):
            self.shape, self.dtype, self.at = torch.Size(shape), dtype, at

        def __getattr__(self, name):
            if name.startswith("__"):
                raise AttributeError(name)
            t = torch.empty(self.shape, dtype=self.dtype, device="meta")
            return dict(get_device=lambda: self.at, data_ptr=lambda: P).get(name, getattr(t, name))

    L.load()
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda device: 0)
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    c = object.__new__(B.KV8Cache)
    c.n_kv_heads, c.head_dim, c.data = 2, 128, OnGpu((10, 2, 128 * 128), u8)
    c._c = cache()
    c._ref = ctypes.addressof(c._c)
    q, table, lens, cu = OnGpu((50, 32, 128), torch.float16), OnGpu((1, 900), i32), OnGpu((1,), i32), OnGpu((2,), i32)
    far, size = OnGpu((1 << 40,), u8, at=1), 64 * 900
    with pytest.raises(ValueError, match="device"):
        c.attention(q, table, lens, cu, 1, size, out=OnGpu(q.shape, torch.float16), workspace=far)
    with pytest.raises(ValueError, match="device"):
        c.accumulate(q, OnGpu((50, 32), f32), table, lens, cu, lens, OnGpu((1, 2, size), f32), 50, size, workspace=far)
    near = OnGpu((16,), u8)                         # of this one: it gets to the library, and is too small
    with pytest.raises(B.WQError, match="workspace of 16 bytes"):
        c.attention(q, table, lens, cu, 1, size, out=OnGpu(q.shape, torch.float16), workspace=near)
    with pytest.raises(B.WQError, match="workspace of 16 bytes"):
        c.accumulate(q, OnGpu((50, 32), f32), table, lens, cu, lens, OnGpu((1, 2, size), f32), 50, size, workspace=near)


def test_rope_wrapper_checks():
    torch = pytest.importorskip("torch")
    q, w = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(64, dtype=torch.float16)
    pos, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    for bad in (dict(q=None, k=None), dict(k=q[:2]), dict(k=q.bfloat16()), dict(k=q[..., :32]), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=None, q_weight=w), dict(k=None, k_weight=w), dict(q_weight=w[:32]),
                dict(inv_freq=f.float()), dict(positions=None)):
        with pytest.raises(ValueError):
            B.wq_qk_norm_rope(**{**dict(q=q, k=q, positions=pos, inv_freq=f), **bad})
