"""The best continuations of many requests' beams: a thin wrapper over the C ABI
(include/bs.h, bs_beam_*).

A decode step of a beam search ends with the choice of the beams that go on,
and the cache's rows follow them:

    beams = Beams(batch, 8, eos=2)
    best = beams.select(logits, scores, done=done)       # logits: a row per beam
    cache.reorder(rows, best.parents.view(-1))
    scores, done, tokens = best.scores, best.done.view(-1), best.tokens.view(-1)

Before the first step a request has one beam: scores of 0 for it and -inf for
the others.  Everything is enqueued on the current (or given) stream and
nothing synchronises.
"""
from __future__ import annotations

import ctypes as C
import threading
from typing import NamedTuple

import torch

from . import _lib as L
from .codec import _capturing, _grown, _on, _same_device, _stream_of


class Best(NamedTuple):
    """The best continuations, (batch, keep) each, best first."""
    scores: torch.Tensor       # float32
    tokens: torch.Tensor       # int32, -1 where there are too few
    parents: torch.Tensor      # int32, rows of the logits, -1 where there are too few
    done: torch.Tensor         # int32, 1 where the token is eos or the parent was done


class Beams:
    """The beams of `batch` requests, and the workspace of their choice."""

    def __init__(self, batch: int, beams: int, keep: int | None = None, eos: int = -1, device: str = "cuda"):
        """keep: how many continuations of a request are kept, by default as
        many as there are beams; eos: the token that ends a beam, if one does."""
        keep = beams if keep is None else keep
        if batch < 0 or not 1 <= beams <= 64 or not 1 <= keep <= 128 or batch * beams > 65535:
            raise ValueError("1 to 64 beams of a request, 65535 in all, of which the best 1 to 128 are kept")
        if not -1 << 31 <= eos < 1 << 31:
            raise ValueError("eos must be a 32-bit token")
        self.batch, self.beams, self.keep, self.eos = batch, beams, keep, eos
        self.device = torch.empty(0, device=device).device
        self._args = L.BeamArgs(batch, beams, keep, 1, L.T_BF16, eos)
        self._ref = C.byref(self._args)
        self._work, self._kept, self._need = None, [], {}
        self._lock = threading.Lock()            # arguments and workspace are one call's until its launches are enqueued

    def select(self, logits: torch.Tensor, scores: torch.Tensor, done: torch.Tensor | None = None, softcap: float = 0.0,
               stream=None) -> Best:
        """The best continuations (bs_beam_select_async): logits (batch *
        beams, vocab) bfloat16 or float32, rows may be strided; scores float32
        and done int32 (not 0: the beam has ended) of batch * beams values.
        softcap c: logits become c tanh(logit / c).  Of equal scores the
        lowest beam comes first, within a beam the larger logit, then the lower
        token.  Calls go on one stream, from any thread."""
        rows, kind = self.batch * self.beams, logits.dtype
        if logits.dim() != 2 or logits.shape[0] != rows or (kind is not torch.bfloat16 and kind is not torch.float32):
            raise ValueError(f"logits must be ({rows}, vocab) bfloat16 or float32")
        vocab = min(logits.shape[1], (1 << 32) - 1)      # the library's 32-bit number would take a larger one's low bits
        if logits.stride(1) != 1 and vocab > 1 and rows:
            raise ValueError("the logits of a beam must be side by side")
        if scores.dtype is not torch.float32 or scores.numel() != rows or not scores.is_contiguous():
            raise ValueError(f"scores must be {rows} contiguous float32 values")
        if done is not None and (done.dtype is not torch.int32 or done.numel() != rows or not done.is_contiguous()):
            raise ValueError(f"done must be {rows} contiguous int32 values")
        if logits.device != self.device or scores.device != self.device or (done is not None and done.device != self.device):
            _same_device(self.device, logits=logits, scores=scores, done=scores if done is None else done)
        with _on(stream):
            got = torch.empty(4, self.batch, self.keep, dtype=torch.int32, device=self.device)
        at, size = got.data_ptr(), 4 * self.batch * self.keep
        with self._lock:
            a = self._args
            a.vocab, a.type, a.softcap = vocab, L.T_FP32 if kind is torch.float32 else L.T_BF16, softcap
            a.row_stride = vocab if rows <= 1 else logits.stride(0)
            a.d_logits, a.d_scores, a.d_done = logits.data_ptr(), scores.data_ptr(), None if done is None else done.data_ptr()
            a.d_scores_out, a.d_tokens, a.d_parents, a.d_done_out = at, at + size, at + 2 * size, at + 3 * size
            need = self._need.get((vocab, kind))
            if need is None:
                need = int(L.lib().bs_beam_work_bytes(self._ref))
                if need:
                    self._need[(vocab, kind)] = need
            w = self._work
            if w is None or w.numel() < need:
                w = self._counted_work(need, stream)
            rc = L.lib().bs_beam_select_async(self._ref, w.data_ptr(), w.numel(), _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_beam_select_async")
        s, t, p, d = got.unbind(0)
        return Best(s.view(torch.float32), t, p, d)

    def _counted_work(self, need: int, stream) -> torch.Tensor:
        """A workspace, its counters zeroed.  Under capture zeroing is recorded
        but not run: the call then has a workspace of its own in the graph's
        memory, zeroed by each replay (a call before the capture spares that)."""
        with _on(stream):
            if _capturing(self.device):
                w = torch.empty(max(need, 4096), dtype=torch.uint8, device=self.device)
                w[:4096].zero_()
                return w
        self._work = _grown(self._work, need, self.device, stream, self._kept, zero=True)
        return self._work
