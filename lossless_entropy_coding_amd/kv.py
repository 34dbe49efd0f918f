"""A paged key/value cache held in 8 bits, and attention over it: thin wrappers
over the C ABI (include/bs.h, bs_kv_*).

One cache serves all layers of a model.  Its rows are sequences; each holds
pages of `page_tokens` tokens, the same page numbers in every layer.  A decode
step extends the rows by one token, then for each layer appends the layer's
keys and values and attends:

    cache = KvCache(layers=42, kv_heads=8, head_dim=256, n_pages=4096, max_seqs=64, max_pages=512)
    cache.extend(rows, ones)
    for layer in range(42):
        cache.append(layer, k, v, rows)
        out = cache.attend(layer, q, rows)

Rows that go on from one prompt (fork) attend together, with the step's plan,
and follow the beams that a search chooses:

    step = KvBatch(cache, rows, groups=groups)
    out = cache.attend_shared(layer, q, step)
    cache.reorder(rows, parents)

Everything is enqueued on the current (or given) stream and nothing
synchronises except check().  The cache keeps its workspaces, so its calls go
on one stream, or on several that wait for each other.  Threads may share a
cache: a call's launches are enqueued together, under the cache's lock.
"""
from __future__ import annotations

import ctypes as C
import threading

import torch

from . import _lib as L
from .codec import _capturing, _grown, _on, _same_device, _stream_of

_INT32, _BF16, _FP32 = torch.int32, torch.bfloat16, torch.float32
_MAX = (1 << 32) - 1             # of the library's 32-bit numbers, which take a larger one's low bits


def _wide(head_dim: int) -> int:
    return -(-head_dim // 64) * 64


class KvCache:
    """A cache (bs_kv_cache) and the tensors that it is made of: k, v, scale,
    refs, table, lens and status."""

    def __init__(self, layers: int, kv_heads: int, head_dim: int, n_pages: int, max_seqs: int, max_pages: int,
                 page_tokens: int = 64, dtype: str = "e4m3", device: str = "cuda"):
        if not 1 <= head_dim <= 256:
            raise ValueError("head_dim goes from 1 to 256")
        z = lambda *shape, t=torch.int32: torch.zeros(*shape, dtype=t, device=device)   # noqa: E731
        wide = _wide(head_dim)
        self._bind(z(layers, n_pages, kv_heads, page_tokens, wide, t=torch.uint8),
                   z(layers, n_pages, kv_heads, wide, page_tokens, t=torch.uint8),
                   z(layers, n_pages, kv_heads, 2, t=torch.float32), z(n_pages), z(max_seqs, max_pages), z(max_seqs),
                   head_dim, dtype)

    @classmethod
    def over(cls, k, v, scale, refs, table, lens, head_dim: int, dtype: str = "e4m3") -> "KvCache":
        """A cache over existing tensors (shapes and types as the constructor's)."""
        self = cls.__new__(cls)
        self._bind(k, v, scale, refs, table, lens, head_dim, dtype)
        return self

    def _bind(self, k, v, scale, refs, table, lens, head_dim, dtype):
        if dtype not in L.KV_TYPES:
            raise ValueError(f"dtype {dtype!r}: one of {', '.join(L.KV_TYPES)}")
        if k.dim() != 5 or not 1 <= head_dim <= 256:
            raise ValueError("k must be (layers, pages, kv_heads, page, wide), head_dim from 1 to 256")
        layers, n_pages, heads, page, wide = k.shape
        want = {"k": (k, torch.uint8, (layers, n_pages, heads, page, _wide(head_dim))),
                "v": (v, torch.uint8, (layers, n_pages, heads, _wide(head_dim), page)),
                "scale": (scale, torch.float32, (layers, n_pages, heads, 2)), "refs": (refs, torch.int32, (n_pages,)),
                "table": (table, torch.int32, (lens.numel(), table.shape[-1])), "lens": (lens, torch.int32, (lens.numel(),))}
        for name, (t, kind, shape) in want.items():
            if t.dtype != kind or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {kind} tensor of shape {shape}")
        _same_device(k.device, **{name: t for name, (t, _, _) in want.items()})
        self.device = k.device
        self.k, self.v, self.scale, self.refs, self.table, self.lens = k, v, scale, refs, table, lens
        self.layers, self.n_pages, self.kv_heads, self.page_tokens = layers, n_pages, heads, page
        self.head_dim, self.dtype, self.max_seqs, self.max_pages = head_dim, dtype, lens.numel(), table.shape[1]
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.c = L.KvCache(layers, n_pages, self.max_seqs, self.max_pages, heads, head_dim, page, L.KV_TYPES[dtype],
                           k.data_ptr(), v.data_ptr(), scale.data_ptr(), refs.data_ptr(), table.data_ptr(),
                           lens.data_ptr(), self.status.data_ptr())
        sizes = L.KvSizes()
        L.check(L.lib().bs_kv_sizes_get(C.byref(self.c), C.byref(sizes)), "bs_kv_sizes_get")
        self.page_bytes = int(sizes.page_bytes)
        self._page_work, self._attend_work, self._kept = None, None, []
        self._ref, self._args = C.byref(self.c), L.KvAttendArgs()
        self._args_ref = C.byref(self._args)
        # the argument block, the workspaces and the table's address are one
        # call's at a time: held until the C call, which lets other threads run,
        # has enqueued its work (and compact has the new table in its place)
        self._lock = threading.Lock()
        self._page_need, self._reorder_need, self._attend_need = {}, {}, {}        # workspace bytes by the sizes of a call

    def _ids(self, t: torch.Tensor, name: str) -> int:
        """Checks a vector of row numbers, counts or offsets; returns its length."""
        if t.dtype is not _INT32 or t.dim() != 1 or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name} must be a contiguous int32 vector on {self.device}")
        return t.numel()

    # ------------------------------------------------------------ pages
    def _work(self, n: int, stream) -> torch.Tensor:
        need = self._page_need.get(n)
        if need is None:
            need = self._page_need[n] = int(L.lib().bs_kv_pages_work_bytes(self._ref, n))
        if self._page_work is None or self._page_work.numel() < need:
            self._page_work = _grown(self._page_work, need, self.device, stream, self._kept)
        return self._page_work

    def extend(self, rows: torch.Tensor, counts: torch.Tensor, stream=None) -> None:
        """Make room for counts[i] more tokens in row rows[i] (distinct rows);
        all rows grow, or none (bs_kv_extend_async)."""
        n = self._ids(rows, "rows")
        if self._ids(counts, "counts") != n:
            raise ValueError("one count per row")
        with self._lock:
            w = self._work(n, stream)
            rc = L.lib().bs_kv_extend_async(self._ref, n, rows.data_ptr(), counts.data_ptr(), w.data_ptr(), w.numel(),
                                            _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_kv_extend_async")

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
        """Empty rows children[i] become copies of rows parents[i], sharing
        their whole pages (bs_kv_fork_async)."""
        n = self._ids(parents, "parents")
        if self._ids(children, "children") != n:
            raise ValueError("one parent per child")
        with self._lock:
            w = self._work(n, stream)
            rc = L.lib().bs_kv_fork_async(self._ref, n, parents.data_ptr(), children.data_ptr(), w.data_ptr(), w.numel(),
                                          _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_kv_fork_async")

    def free(self, rows: torch.Tensor, stream=None) -> None:
        """Empty rows (bs_kv_free_async)."""
        n = self._ids(rows, "rows")
        with self._lock:
            rc = L.lib().bs_kv_free_async(self._ref, n, rows.data_ptr(), _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_kv_free_async")

    def reorder(self, rows: torch.Tensor, parents: torch.Tensor, stream=None) -> None:
        """Rows rows[i] (distinct) take the tokens of rows[parents[i]], all at
        once (-1: the row becomes empty); whole pages are shared
        (bs_kv_reorder_async).  After a choice of beams, parents are its
        Best.parents where the rows are in the order of the logits."""
        n = self._ids(rows, "rows")
        if self._ids(parents, "parents") != n:
            raise ValueError("one parent per row")
        with self._lock:
            need = self._reorder_need.get(n)
            if need is None:
                need = self._reorder_need[n] = int(L.lib().bs_kv_reorder_work_bytes(self._ref, n))
            w = self._page_work
            if w is None or w.numel() < need:
                w = self._page_work = _grown(w, need, self.device, stream, self._kept)
            rc = L.lib().bs_kv_reorder_async(self._ref, n, rows.data_ptr(), parents.data_ptr(), w.data_ptr(), w.numel(),
                                             _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_kv_reorder_async")

    def copy_pages(self, source: torch.Tensor, target: torch.Tensor, stream=None) -> None:
        """Copy pages in every layer (bs_kv_copy_pages_async)."""
        n = self._ids(source, "source")
        if self._ids(target, "target") != n:
            raise ValueError("one target per source")
        with self._lock:
            L.check(L.lib().bs_kv_copy_pages_async(self._ref, n, source.data_ptr(), target.data_ptr(),
                                                   _stream_of(self.device, stream)), "bs_kv_copy_pages_async")

    def compact(self, table_out: torch.Tensor | None = None, refs_out: torch.Tensor | None = None, stream=None) -> None:
        """Move the pages in use to the lowest places (bs_kv_compact_async).
        With table_out and refs_out the new table and counts go there and the
        cache keeps its own; without, the cache goes on with the new ones in
        tensors of its own, kept for the next time (a captured graph goes on
        with those it was captured with: capture it again)."""
        if (table_out is None) != (refs_out is None):
            raise ValueError("table_out and refs_out go together")
        with self._lock:
            swap = table_out is None
            if swap:
                if getattr(self, "_spare", None) is None:
                    with _on(stream):
                        self._spare = (torch.empty_like(self.table), torch.empty_like(self.refs))
                table_out, refs_out = self._spare
            for t, like, name in ((table_out, self.table, "table_out"), (refs_out, self.refs, "refs_out")):
                if t.dtype != like.dtype or t.shape != like.shape or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(like.shape)}")
            _same_device(self.device, table_out=table_out, refs_out=refs_out)
            w = self._work(0, stream)
            L.check(L.lib().bs_kv_compact_async(self._ref, table_out.data_ptr(), refs_out.data_ptr(), w.data_ptr(), w.numel(),
                                                _stream_of(self.device, stream)), "bs_kv_compact_async")
            if swap:
                self._spare = (self.table, self.refs)
                self.table, self.refs = table_out, refs_out
                self.c.d_table, self.c.d_refs = table_out.data_ptr(), refs_out.data_ptr()

    # ------------------------------------------------------------ tokens
    def _tokens(self, t: torch.Tensor, heads: int | None, name: str) -> int:
        """Checks a (tokens, heads, head_dim) tensor with a token's values side
        by side; returns its token stride."""
        shape = t.shape
        if len(shape) != 3 or shape[2] != self.head_dim or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} must be (tokens, {heads or 'heads'}, {self.head_dim})")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        n, h, d = shape
        if t.is_contiguous():
            return h * d
        s = t.stride()
        if n and ((d > 1 and s[2] != 1) or (h > 1 and s[1] != d)):
            raise ValueError(f"the values of a token must be side by side in {name}")
        return h * d if n <= 1 else s[0]

    def _rows(self, rows, starts, total, max_new):
        n = self._ids(rows, "rows")
        if starts is None:
            if n != total:
                raise ValueError(f"{total} tokens for {n} rows: give starts")
            return n, 1, None
        if self._ids(starts, "starts") != n + 1:
            raise ValueError("starts holds one offset per row and the end")
        return n, max(1, min(total, total if max_new is None else max_new)), starts.data_ptr()

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, rows: torch.Tensor, starts: torch.Tensor | None = None,
               max_new: int | None = None, stream=None) -> None:
        """Store the keys and values of the rows' last tokens
        (bs_kv_append_async): k and v (tokens, kv_heads, head_dim) bfloat16 or
        float32, tokens starts[i] .. starts[i + 1] - 1 of row rows[i] (without
        starts one each); max_new: the most of one row, if it is known."""
        kind = k.dtype
        if v.dtype is not kind or (kind is not _BF16 and kind is not _FP32) or k.shape != v.shape:
            raise ValueError("k and v must have one shape and be bfloat16 or float32")
        ks, vs, total = self._tokens(k, self.kv_heads, "k"), self._tokens(v, self.kv_heads, "v"), k.shape[0]
        n, most, at = self._rows(rows, starts, total, max_new)
        with self._lock:
            rc = L.lib().bs_kv_append_async(self._ref, layer if 0 <= layer < _MAX else _MAX, n, rows.data_ptr(), at, total, most, k.data_ptr(),
                                            ks, v.data_ptr(), vs, L.T_FP32 if kind is _FP32 else L.T_BF16, _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_kv_append_async")

    def attend(self, layer: int, q: torch.Tensor, rows: torch.Tensor, starts: torch.Tensor | None = None,
               max_new: int | None = None, max_len: int = 0, scale: float = 0.0, window: int = 0, sinks: int = 0,
               softcap: float = 0.0, out: torch.Tensor | None = None, lse: bool | torch.Tensor = False, stream=None):
        """Attention of the rows' last tokens over all that they see
        (bs_kv_attend_async): q (tokens, heads, head_dim) bfloat16, tokens as in
        append.  window: 0 or how many of the last tokens a query sees, besides
        the first `sinks`; softcap c: logits become c tanh(logit / c); scale 0:
        1 / sqrt(head_dim).  max_len: how long the rows are at most, if it is
        known (it decides how the work is split, not the result).  Returns
        the result (q's shape, bfloat16), and with lse the logarithms of the
        softmax sums (tokens, heads) as float32."""
        total, heads, qs, os, out, lse, window, sinks, max_len = self._results(q, out, lse, window, sinks, max_len, stream)
        n, most, at = self._rows(rows, starts, total, max_new)
        with self._lock:
            a = self._args
            a.layer, a.n_seqs, a.heads = layer if 0 <= layer < _MAX else _MAX, n, heads
            a.total_q, a.max_new, a.max_len = total, most, max_len
            a.d_seqs, a.d_starts, a.d_q, a.d_out = rows.data_ptr(), at, q.data_ptr(), out.data_ptr()
            a.d_lse = None if lse is False else lse.data_ptr()
            a.q_stride, a.out_stride, a.scale, a.softcap, a.window, a.sinks = qs, os, scale, softcap, window, sinks
            sizes = (n, heads, total, most, max_len, window, sinks)
            need = self._attend_need.get(sizes)
            known = need is not None
            if not known:
                need = int(L.lib().bs_kv_attend_work_bytes(self._ref, self._args_ref))
            w = self._attend_work
            if need and (w is None or w.numel() < need):
                w = self._counted_work(need, stream)
            rc = L.lib().bs_kv_attend_async(self._ref, self._args_ref, w.data_ptr() if need else None, need,
                                            _stream_of(self.device, stream))
            if not rc and not known:                       # a refused call's size is 0, whatever its rows need
                if len(self._attend_need) > 4096:          # lengths that grow token by token
                    self._attend_need.clear()
                self._attend_need[sizes] = need
        if rc:
            L.check(rc, "bs_kv_attend_async")
        return out if lse is False else (out, lse)

    def attend_shared(self, layer: int, q: torch.Tensor, batch: "KvBatch", scale: float = 0.0, window: int = 0, sinks: int = 0,
                      softcap: float = 0.0, out: torch.Tensor | None = None, lse: bool | torch.Tensor = False, stream=None):
        """attend of the tokens of a plan, reading the tokens that the rows of
        a group have in common once for all of them
        (bs_kv_attend_shared_async): q (batch.total, heads, head_dim) in the
        plan's order; the other arguments and the results are attend's.  The
        plan is this cache's and holds until its rows change.  Where
        batch.max_new x heads / kv_heads is 64 or more it is attend itself, so
        a plan with counts should say its max_new.  Where little is read attend
        is faster, since it takes one launch: by up to 1.2 us (2.4 outside a
        graph) where rows x kv_heads x length / 64 is below about 500, and for
        rows of up to some 150 tokens by 1.4 us (few rows) to 8 (64 rows)."""
        if batch.cache is not self:
            raise ValueError("the plan is another cache's")
        total, heads, qs, os, out, lse, window, sinks, max_len = self._results(q, out, lse, window, sinks, batch.max_len, stream)
        if total != batch.total:
            raise ValueError(f"{total} tokens, {batch.total} in the plan")
        with self._lock:
            a = self._args
            a.layer, a.heads, a.max_len = layer if 0 <= layer < _MAX else _MAX, heads, max_len
            a.d_q, a.d_out, a.d_lse = q.data_ptr(), out.data_ptr(), None if lse is False else lse.data_ptr()
            a.q_stride, a.out_stride, a.scale, a.softcap, a.window, a.sinks = qs, os, scale, softcap, window, sinks
            sizes = (batch.n, batch.n_groups, heads, total, batch.max_new, max_len, window, sinks)
            need = self._attend_need.get(sizes)
            known = need is not None
            if not known:
                need = int(L.lib().bs_kv_attend_shared_work_bytes(self._ref, self._args_ref, batch.ref))
            w = self._attend_work
            if need and (w is None or w.numel() < need):
                w = self._counted_work(need, stream)
            rc = L.lib().bs_kv_attend_shared_async(self._ref, self._args_ref, batch.ref, w.data_ptr() if need else None, need,
                                                   _stream_of(self.device, stream))
            if not rc and not known:
                if len(self._attend_need) > 4096:
                    self._attend_need.clear()
                self._attend_need[sizes] = need
        if rc:
            L.check(rc, "bs_kv_attend_shared_async")
        return out if lse is False else (out, lse)

    def _results(self, q, out, lse, window, sinks, max_len, stream):
        """Checks of what attention reads and writes, and memory for its results."""
        if q.dtype is not _BF16:
            raise ValueError("q must be bfloat16")
        qs = os = self._tokens(q, None, "q")
        shape = q.shape
        if out is None:
            with _on(stream):
                out = torch.empty(shape, dtype=_BF16, device=self.device)
            os = shape[1] * self.head_dim
        elif out.dtype is not _BF16 or out.shape != shape:
            raise ValueError("out must be bfloat16 of q's shape")
        else:
            os = self._tokens(out, None, "out")
        if lse is True:
            with _on(stream):
                lse = torch.empty(shape[:2], dtype=_FP32, device=self.device)
        elif lse is not False and (lse.dtype is not _FP32 or lse.shape != shape[:2] or not lse.is_contiguous() or
                                   lse.device != self.device):
            raise ValueError(f"lse must be a contiguous float32 tensor of (tokens, heads) on {self.device}")
        if window < 0 or sinks < 0 or max_len < 0:
            raise ValueError("window, sinks and max_len are not negative")
        # rows are shorter than the largest numbers that the library takes
        return shape[0], shape[1], qs, os, out, lse, min(window, _MAX), min(sinks, _MAX), min(max_len, _MAX)

    def _counted_work(self, need: int, stream) -> torch.Tensor:
        """A workspace for attend, its counters zeroed.  Under capture zeroing
        is recorded but not run, so no other call may count on it: the call
        then has a workspace of its own in the graph's memory, whose counters
        each replay zeroes first (a call before the capture spares that)."""
        with _on(stream):
            if _capturing(self.device):
                w = torch.empty(need, dtype=torch.uint8, device=self.device)
                w[:4096].zero_()
                return w
        self._attend_work = _grown(self._attend_work, need, self.device, stream, self._kept, zero=True)
        return self._attend_work

    def check(self) -> None:
        """Raise if a call met one of the conditions that bs.h lists, and clear
        it; synchronises."""
        bits = int(self.status.item())
        if bits:
            self.status.zero_()
            raise RuntimeError("key/value cache: " + "; ".join(v for b, v in L.KV_STATUS.items() if bits & b))


class KvBatch:
    """The plan of a step's tokens (bs_kv_batch), made once a step, after
    extend, for all layers.  Row rows[i] of the cache has counts[i] new tokens
    (without counts one each), its last ones, side by side in the step's
    tensors; groups: offsets into rows of the runs of rows that go on from one
    prompt (without: one group of all rows).  A row that has fewer than 64
    tokens in common with its group's first one, as a beam that was emptied and
    grows anew, stands alone in attention; the others go on together if they
    are two at least and half of the group.

    starts (rows + 1), places and slots (tokens; int64 slots), table (rows,
    pages of max_len), lead and shared (rows) are int32 tensors on the device
    as bs.h describes them, written by the call and each update().  append and
    attend take `starts`, a rotary embedding `places`, kernels of one's own
    `slots` and `table`, and KvCache.attend_shared all of it."""

    def __init__(self, cache: KvCache, rows: torch.Tensor, counts: torch.Tensor | None = None, groups: torch.Tensor | None = None,
                 total: int | None = None, max_new: int | None = None, max_len: int = 0, stream=None):
        """total: tokens in all, needed with counts; max_new: the most of one
        row, if it is known; max_len: how long the rows are at most (0: as the
        cache allows), which decides the width of table."""
        n = rows.numel()
        if counts is None:
            total, max_new = n if total is None else total, 1 if max_new is None else max_new
        elif total is None:
            raise ValueError("with counts the number of tokens must be given (total)")
        if not 0 <= total < 1 << 31 or max_len < 0:
            raise ValueError("total goes from 0 to 2^31 - 1, max_len is not negative")
        self.cache, self.n, self.total = cache, n, total
        self.max_new = max(1, min(total, total if max_new is None else max_new))
        self.n_groups = 1 if groups is None else max(groups.numel() - 1, 0)
        self.max_len = min(max_len or cache.max_pages * cache.page_tokens, cache.max_pages * cache.page_tokens)
        width = -(-self.max_len // cache.page_tokens)
        self._counted = counts is not None
        sizes = [4 + 8 * (self.n_groups + n), 2 * total, n + 1, total, n * width, n, n, n]
        with _on(stream):        # zeroed: the plan's counter is 0 before its first call
            info, slots, self.starts, self.places, table, self.lead, self.shared, self.rows = \
                torch.zeros(sum(sizes), dtype=_INT32, device=cache.device).split(sizes)
        self.slots, self.table = slots.view(torch.int64), table.view(n, width)
        self.c = L.KvBatch(n, self.n_groups, total, self.max_new, width, 0, self.rows.data_ptr(), self.starts.data_ptr(),
                           self.places.data_ptr(), slots.data_ptr(), table.data_ptr(), self.lead.data_ptr(),
                           self.shared.data_ptr(), info.data_ptr())
        self._info, self.ref = info, C.byref(self.c)
        self.update(rows, counts, groups, stream)

    def update(self, rows: torch.Tensor, counts: torch.Tensor | None = None, groups: torch.Tensor | None = None, stream=None) -> None:
        """The plan of another step with as many rows, tokens and groups
        (bs_kv_batch_async); the buffers stay, as a captured graph needs."""
        cache = self.cache
        if cache._ids(rows, "rows") != self.n:
            raise ValueError(f"{self.n} rows")
        if (counts is not None) != self._counted or (counts is not None and cache._ids(counts, "counts") != self.n):
            raise ValueError("one count per row" if self._counted else "a plan made without counts has one token per row")
        if (1 if groups is None else cache._ids(groups, "groups") - 1) != self.n_groups:
            raise ValueError(f"offsets of {self.n_groups} groups")
        with cache._lock:
            rc = L.lib().bs_kv_batch_async(cache._ref, self.ref, rows.data_ptr(), None if counts is None else counts.data_ptr(),
                                           None if groups is None else groups.data_ptr(), _stream_of(cache.device, stream))
        if rc:
            L.check(rc, "bs_kv_batch_async")
