"""The paged 8-bit key/value cache on the GPU (include/wq.h, "8-bit key/value
cache"): written and read as the 4-bit one (``kv4``), with the same
``wq_kv4_plan``.  A decode step that evicts from time to time is

    wq_kv4_plan(lens, cu_rows, block_table, free_pages, new_lens, slots, runs, taken)
    cache.append(k, v, slots, runs)
    out = cache.attention(q, block_table, new_lens, cu_rows, max_rows, max_len, lse=lse)
    cache.accumulate(q, lse, block_table, new_lens, cu_rows, lens, mass, max_rows, max_len)
    cache.evict(mass, block_table, new_lens, keep, recent, free_pages, new_table, ...)

Everything but the sizes is device data.  Calls are made on the current device; one
with ``stream`` runs there: what it reads has to be ready on that stream, and its result
is to be awaited there.
"""

from __future__ import annotations

import ctypes

from . import _lib as L
from .kv4 import KV4Cache, _dtype, _new, _strided, _workspace


def _f32(t, shape, what):
    """Pointer of a contiguous float32 GPU tensor of the given shape."""
    import torch
    if t.dtype is torch.float32 and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous GPU tensor, float32 {list(shape)}: got {t.dtype} {list(t.shape)}")


def _same_device(*tensors):
    """All on the current device: the launches go there."""
    now = L._current_device()
    for t in tensors:
        if t.get_device() != now:
            raise ValueError(f"a tensor on {t.device}, the current device is {now}")


def _zeros(n, device, stream):
    """n int32 zeros that only a call on `stream` uses."""
    import torch
    if stream is None:
        return torch.zeros(n, dtype=torch.int32, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(n, dtype=torch.int32, device=device)


class KV8Cache:
    """data uint8 [n_pages, n_kv_heads, 128 D] and exponents int8 [n_pages,
    n_kv_heads, 8], as plain device buffers."""

    def __init__(self, data, exponents):
        import torch
        if data.dtype != torch.uint8 or data.dim() != 3 or data.shape[2] % 128:
            raise ValueError("data must be uint8 [n_pages, n_kv_heads, 128 D]")
        self.data, self.exponents = data, exponents
        n, h, size = data.shape
        self.n_pages, self.n_kv_heads, self.head_dim = n, h, size // 128
        if exponents.dtype != torch.int8 or exponents.shape != (n, h, 8) or exponents.device != data.device:
            raise ValueError("exponents must be int8 [n_pages, n_kv_heads, 8] beside the data")
        self._c = L.Kv8Cache(L._dptr(data), L._dptr(exponents), self.n_pages, self.n_kv_heads,
                             self.head_dim)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, device="cuda") -> "KV8Cache":
        import torch
        return cls(torch.zeros((n_pages, n_kv_heads, 128 * head_dim), dtype=torch.uint8, device=device),
                   torch.zeros((n_pages, n_kv_heads, 8), dtype=torch.int8, device=device))

    def append(self, k, v, slots, runs, stream=None):
        """Writes k, v [rows, n_kv_heads, D] (FP16 or BF16, any row and head
        strides that are multiples of 8) into their slots."""
        fn = L.load().wq_kv8_append
        T = slots.numel()
        want = (T, self.n_kv_heads, self.head_dim)
        if k.shape != want or v.shape != want or k.dtype != v.dtype:
            raise ValueError(f"k and v must be {list(want)} of one type")
        kp, kr, kh = _strided(k, "k")
        vp, vr, vh = _strided(v, "v")
        _same_device(self.data, k, v, slots, runs)
        L._check(fn(self._ref, _dtype(k), kp, kr, kh, vp, vr, vh, T, L._i32(slots, (T,), "slots"),
                    L._i32(runs, (runs.shape[0], 2), "runs"), runs.shape[0], L._stream(stream)))

    _rows = KV4Cache._rows

    def attention(self, q, block_table, lens, cu_rows, max_rows, max_len, scale=None, window=0,
                  out=None, lse=None, workspace=None, stream=None):
        """Attention of q [rows, n_heads, D] over the cached tokens of its
        sequences (lens counts the rows' own), over the last `window` of each row
        if that is not 0.  lse float32 [rows, n_heads] receives the logarithm of the
        softmax sums.  Rows behind the last of cu_rows are left as they are.  Decodes beside
        a long piece of a prompt are faster in a call of their own."""
        lib = L.load()
        a = self._rows(q, block_table, lens, cu_rows)
        _same_device(self.data, q, block_table, lens, cu_rows)
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != q.get_device():
            raise ValueError("out must have q's shape, type and device")
        lp = None
        if lse is not None:
            lp = _f32(lse, q.shape[:2], "lse")
            _same_device(lse)
        ar = ctypes.addressof(a)
        need = lib.wq_kv8_attention_workspace(self._ref, ar, max_rows, max_len)
        if need < 0:
            L._check(need)
        if workspace is not None:
            _same_device(workspace)
        elif need:
            workspace = _workspace(need, q.device, stream)
        L._check(lib.wq_kv8_attention(
            self._ref, ar, max_rows, max_len, self.head_dim ** -0.5 if scale is None else scale, window,
            L._dptr(out), lp, L._dptr(workspace),
            0 if workspace is None else workspace.numel(), L._stream(stream)))
        return out

    def accumulate(self, q, lse, block_table, lens, cu_rows, held, mass, max_rows, max_len, scale=None,
                   window=0, workspace=None, stream=None):
        """Adds to mass float32 [sequences, n_kv_heads, tokens] the softmax weights that
        the rows and heads give each cached token; lse is attention's for the same
        arguments, held int32 [sequences] how many tokens have a mass already (the
        others start from 0, also where there are no rows).  Returns mass."""
        lib = L.load()
        a = self._rows(q, block_table, lens, cu_rows)
        _same_device(self.data, q, lse, block_table, lens, cu_rows, held, mass)
        if mass.dim() != 3:
            raise ValueError("mass must be float32 [sequences, n_kv_heads, tokens]")
        mp = _f32(mass, (a.n_seqs, self.n_kv_heads, mass.shape[2]), "mass")
        lp = _f32(lse, (a.n_rows, a.n_heads), "lse")
        if not a.n_rows and a.n_seqs:
            # no rows: the call does nothing, and a padded batch of one row behind the last
            # sequence, which is never read, starts the new tokens' masses
            none = _zeros(max(a.n_seqs + 1, 4), q.device, stream)
            lp = a.q = a.cu_rows = none.data_ptr()
            a.n_rows, a.q_row_stride, a.q_head_stride, workspace = 1, 0, 0, None
        ar = ctypes.addressof(a)
        need = lib.wq_kv8_accumulate_workspace(self._ref, ar, max_rows, max_len)
        if need < 0:
            L._check(need)
        if workspace is not None:
            _same_device(workspace)
        elif need:
            workspace = _workspace(need, q.device, stream)
        L._check(lib.wq_kv8_accumulate(
            self._ref, ar, max_rows, max_len, lp, self.head_dim ** -0.5 if scale is None else scale, window,
            L._i32(held, (a.n_seqs,), "held"), mp, mass.shape[2], L._dptr(workspace),
            0 if workspace is None else workspace.numel(), L._stream(stream)))
        return mass

    def evict(self, mass, block_table, lens, keep, recent, free_pages, new_table, new_lens, new_mass,
              taken, kept=None, stream=None):
        """Moves the last `recent` tokens and those of most mass, `keep` in all, of
        every sequence that is longer to the next pages of free_pages: new_table
        (block_table's shape), new_lens and new_mass [sequences, n_kv_heads, at least
        keep] are the sequences' new ones, taken [1] the pages taken.  The old pages
        stay as they are.  Returns kept int32 [sequences, n_kv_heads, keep], the
        tokens kept, -1 past the end."""
        import torch
        lib = L.load()
        B, width = block_table.shape
        H, F = self.n_kv_heads, free_pages.numel()
        if mass.dim() != 3 or new_mass.dim() != 3:
            raise ValueError("masses must be float32 [sequences, n_kv_heads, tokens]")
        _same_device(self.data, mass, block_table, lens, free_pages, new_table, new_lens, new_mass, taken)
        if kept is None:
            kept = _new((B, H, keep), torch.int32, mass.device, stream)
        _same_device(kept)
        L._check(lib.wq_kv8_evict(
            self._ref, _f32(mass, (B, H, mass.shape[2]), "mass"), mass.shape[2],
            L._i32(block_table, (B, width), "block_table"), width, L._i32(lens, (B,), "lens"), B, keep, recent,
            L._i32(free_pages, (F,), "free_pages"), F, L._i32(new_table, (B, width), "new_table"),
            L._i32(new_lens, (B,), "new_lens"), _f32(new_mass, (B, H, new_mass.shape[2]), "new_mass"),
            new_mass.shape[2], L._i32(taken, (1,), "taken"), L._i32(kept, (B, H, keep), "kept"),
            L._stream(stream)))
        return kept
