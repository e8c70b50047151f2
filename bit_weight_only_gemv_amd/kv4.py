"""The paged 4-bit key/value cache on the GPU and the calls that write and read
it (include/wq.h, "4-bit key/value cache").  A decode step is

    wq_kv4_plan(lens, cu_rows, block_table, free_pages, new_lens, slots, runs, taken)
    cache.append(k, v, slots, runs)
    out = cache.attention(q, block_table, new_lens, cu_rows, max_rows, max_len)

or, for long sequences, with ``sel = cache.select(q, block_table, new_lens,
cu_rows, n_sel)`` passed to ``attention``.  Everything but the sizes is device
data, so a captured graph of the step serves other lengths too; it is fastest near
the max_len that it was captured with.  A call with ``stream`` runs there: what it
reads has to be ready on that stream, and its result is to be awaited there.
"""

from __future__ import annotations

import ctypes

from . import _lib as L


_TYPES = {"torch.float16": L.WQ_DT_F16, "torch.bfloat16": L.WQ_DT_BF16}


def _dtype(t):
    d = _TYPES.get(t.dtype)
    if d is None:                       # by name the first time, then by type
        d = _TYPES.get(str(t.dtype))
        if d is None:
            raise ValueError(f"float16 or bfloat16 expected, got {t.dtype}")
        _TYPES[t.dtype] = d
    return d


def _strided(t, what):
    """(pointer, row stride, head stride) of a GPU tensor [rows, heads, D]."""
    if not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{what} must be a GPU tensor [rows, heads, D]")
    r, h, c = t.stride()
    if c != 1 and t.numel():
        raise ValueError(f"{what}: channels must be consecutive")
    if (r | h) & 7:                     # the stride of a single row or head is never used
        rows, heads, _ = t.shape
        r, h = r if rows > 1 else 0, h if heads > 1 else 0
    return t.data_ptr(), r, h


def _new(shape, dtype, device, stream):
    """A tensor that a call on `stream` writes and the current stream's work uses.
    It is memory of `stream`, not of the current one, whose last user there may not
    be done; and it is not handed out again before the current stream's work that
    is queued when it is dropped."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    t = _of_stream(shape, dtype, device, stream)
    if t.numel():
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _workspace(nbytes, device, stream):
    """Memory that only a call on `stream` uses."""
    import torch
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return _of_stream(nbytes, torch.uint8, device, stream)


def _of_stream(shape, dtype, device, stream):
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class KV4Cache:
    """data uint8 [n_pages, n_kv_heads, 80 D] and summary float16 [n_pages,
    n_kv_heads, 2, D] (None: no page selection), as plain device buffers."""

    def __init__(self, data, summary=None):
        import torch
        if data.dtype != torch.uint8 or data.dim() != 3 or data.shape[2] % 80:
            raise ValueError("data must be uint8 [n_pages, n_kv_heads, 80 D]")
        self.data, self.summary = data, summary
        self.n_pages, self.n_kv_heads, self.head_dim = data.shape[0], data.shape[1], data.shape[2] // 80
        if summary is not None and (summary.dtype != torch.float16 or tuple(summary.shape) != (
                self.n_pages, self.n_kv_heads, 2, self.head_dim)):
            raise ValueError("summary must be float16 [n_pages, n_kv_heads, 2, D]")
        self._c = L.Kv4Cache(L._dptr(data), L._dptr(summary), self.n_pages, self.n_kv_heads,
                             self.head_dim)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, summary: bool = True,
              device="cuda") -> "KV4Cache":
        import torch
        data = torch.zeros((n_pages, n_kv_heads, 80 * head_dim), dtype=torch.uint8, device=device)
        sm = torch.zeros((n_pages, n_kv_heads, 2, head_dim), dtype=torch.float16,
                         device=device) if summary else None
        return cls(data, sm)

    def append(self, k, v, slots, runs, stream=None):
        """Writes k, v [rows, n_kv_heads, D] (FP16 or BF16, any row and head
        strides that are multiples of 8) into their slots."""
        fn = L.load().wq_kv4_append
        T = slots.numel()
        want = (T, self.n_kv_heads, self.head_dim)
        if k.shape != want or v.shape != want or k.dtype != v.dtype:
            raise ValueError(f"k and v must be {list(want)} of one type")
        kp, kr, kh = _strided(k, "k")
        vp, vr, vh = _strided(v, "v")
        L._check(fn(self._ref, _dtype(k), kp, kr, kh, vp, vr, vh, T, L._i32(slots, (T,), "slots"),
                    L._i32(runs, (runs.shape[0], 2), "runs"), runs.shape[0], L._stream(stream)))

    def _rows(self, q, block_table, lens, cu_rows):
        B, width = block_table.shape
        T, H, D = q.shape
        if D != self.head_dim:
            raise ValueError(f"q has {D} channels, the cache {self.head_dim}")
        if T and not B:
            raise ValueError(f"{T} rows of no sequences")
        p, r, h = _strided(q, "q")
        return L.Kv4Rows(L._i32(block_table, (B, width), "block_table"), L._i32(lens, (B,), "lens"),
                         L._i32(cu_rows, (B + 1,), "cu_rows"), width, B, T, H, _dtype(q), p, r, h)

    def select(self, q, block_table, lens, cu_rows, n_sel, sel=None, workspace=None, stream=None):
        """Positions in the block table of the n_sel pages of highest bound for
        each row and key/value head: int32 [rows, n_kv_heads, n_sel], rising,
        -1 past the end."""
        import torch
        lib = L.load()
        a = self._rows(q, block_table, lens, cu_rows)
        shape = (a.n_rows, self.n_kv_heads, n_sel)
        if sel is None:
            sel = _new(shape, torch.int32, q.device, stream)
        need = lib.wq_kv4_select_workspace(a.n_rows, self.n_kv_heads, a.table_width)
        if need < 0:
            L._check(need)
        if workspace is None:
            workspace = _workspace(need, q.device, stream)
        L._check(lib.wq_kv4_select(self._ref, ctypes.addressof(a), n_sel, L._i32(sel, shape, "sel"),
                                   L._dptr(workspace), workspace.numel(), L._stream(stream)))
        return sel

    def attention(self, q, block_table, lens, cu_rows, max_rows, max_len, scale=None, window=0,
                  sel=None, out=None, lse=None, workspace=None, stream=None):
        """Attention of q [rows, n_heads, D] over the cached tokens of its
        sequences (lens counts the rows' own), over those in the pages of sel if
        given, over the last `window` of each row if that is not 0.  lse float32
        [rows, n_heads] receives the logarithm of the softmax sums."""
        import torch
        lib = L.load()
        n_sel = 0 if sel is None else sel.shape[-1]
        if sel is not None and n_sel == 0:      # its NULL pointer would mean all tokens
            raise ValueError("sel has no places")
        a = self._rows(q, block_table, lens, cu_rows)
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        elif out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and type")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2]):
            raise ValueError("lse must be float32 [rows, n_heads]")
        if scale is None:
            scale = self.head_dim ** -0.5
        ar = ctypes.addressof(a)
        need = lib.wq_kv4_attention_workspace(self._ref, ar, max_rows, max_len, n_sel)
        if need < 0:
            L._check(need)
        if workspace is None and need:
            workspace = _workspace(need, q.device, stream)
        L._check(lib.wq_kv4_attention(
            self._ref, ar, max_rows, max_len, scale, window,
            None if sel is None else L._i32(sel, (a.n_rows, self.n_kv_heads, n_sel), "sel"), n_sel,
            L._dptr(out), L._dptr(lse), L._dptr(workspace),
            0 if workspace is None else workspace.numel(), L._stream(stream)))
        return out
