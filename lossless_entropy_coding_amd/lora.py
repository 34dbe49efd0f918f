"""Low-rank adapters of many requests beside a shared projection: thin wrappers
over the C ABI (include/bs.h, bs_lora_*).

    y[t] += s_a B_a (A_a x_t),   a = the adapter of token t

A LoraPack holds every adapter of one projection, laid out once; a LoraBatch
says which token has which adapter and is made once per step, for all
projections that the step's tokens go through.  Beside a projection in the
fixed-width form, codec.FixedPlan.gemm_lora computes both products together;
LoraPack.add adds the adapters' part to a projection made elsewhere.
"""
from __future__ import annotations

import ctypes as C
import threading

import torch

from . import _lib as L
from .codec import _grown, _on, _same_device, _stream_of


class LoraPack:
    """All adapters of one projection in device memory."""

    def __init__(self, adapters, device: str = "cuda"):
        """adapters: a list of (A, B, s): A (r, cols) and B (rows, r) tensors,
        taken in bfloat16, and a number; r from 1 to 128, each adapter its own."""
        if not adapters:
            raise ValueError("no adapters")
        rows, cols = int(adapters[0][1].shape[0]), int(adapters[0][0].shape[1])
        ranks = []
        for a, b, _ in adapters:
            if a.dim() != 2 or b.dim() != 2 or a.shape[1] != cols or b.shape[0] != rows or a.shape[0] != b.shape[1]:
                raise ValueError(f"an adapter of a {rows} x {cols} projection has A (r, {cols}) and B ({rows}, r)")
            ranks.append(int(a.shape[0]))
        if not 1 <= min(ranks) or max(ranks) > 128:
            raise ValueError("ranks go from 1 to 128")
        self.rows, self.cols, self.adapters = rows, cols, len(adapters)
        self.rank = next(r for r in (16, 32, 64, 128) if r >= max(ranks))
        steps = -(-cols // 32)
        rows_of_a = torch.zeros(len(adapters), self.rank, 32 * steps, dtype=torch.bfloat16, device=device)
        self.b = torch.zeros(len(adapters), rows, self.rank, dtype=torch.bfloat16, device=device)
        for i, (a, b, _) in enumerate(adapters):
            rows_of_a[i, :ranks[i], :cols] = a
            self.b[i, :, :ranks[i]] = b
        # the operand order of bs.h: (adapter, 16 rows, 32 columns, lane group, row, 8 columns)
        self.a = rows_of_a.view(len(adapters), self.rank // 16, 16, steps, 4, 8).permute(0, 1, 3, 4, 2, 5).contiguous()
        self.ranks = torch.tensor(ranks, dtype=torch.int32, device=device)
        self.factor = torch.tensor([float(s) for _, _, s in adapters], dtype=torch.float32, device=device)
        self.device = self.a.device
        self.c = L.LoraPack(self.adapters, self.rank, rows, cols, self.a.data_ptr(), self.b.data_ptr(),
                            self.ranks.data_ptr(), self.factor.data_ptr())
        self.ref = C.byref(self.c)
        self._work, self._kept, self._need = None, [], {}
        self._lock = threading.Lock()            # the workspace is one call's until its launches are enqueued

    def work_bytes(self, tokens: int) -> int:
        """Workspace of add() for this many tokens (bs_lora_work_bytes)."""
        need = self._need.get(tokens)
        if need is None:
            need = self._need[tokens] = int(L.lib().bs_lora_work_bytes(self.ref, tokens))
        return need

    def add(self, y: torch.Tensor, x: torch.Tensor, batch: "LoraBatch", out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
        """y plus each token's adapter (bs_lora_add_async): x (tokens, cols)
        bfloat16, y (tokens, rows) float32 or bfloat16; rows of x and y may be
        strided.  Written to `out` (y's shape, type and strides), by default y
        itself.  The pack keeps the workspace: calls go on one stream, from any
        thread."""
        out = y if out is None else out
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.cols or (x.shape[0] and x.stride(1) != 1):
            raise ValueError(f"x must be a (tokens, {self.cols}) bfloat16 tensor with adjacent columns")
        if y.dtype not in (torch.float32, torch.bfloat16) or tuple(y.shape) != (x.shape[0], self.rows) or \
                (x.shape[0] and y.stride(1) != 1 and self.rows > 1):
            raise ValueError(f"y must be a ({x.shape[0]}, {self.rows}) float32 or bfloat16 tensor with adjacent rows")
        if out.dtype != y.dtype or out.shape != y.shape or out.stride() != y.stride():
            raise ValueError("out must have y's shape, type and strides")
        batch.check_for(self, x.shape[0])
        if x.device != self.device or y.device != self.device or out.device != self.device or batch.dev.device != self.device:
            _same_device(self.device, x=x, y=y, out=out, batch=batch.dev)
        if x.shape[0] == 0:
            return out
        with self._lock:
            need = self.work_bytes(x.shape[0])
            if self._work is None or self._work.numel() < need:
                self._work = _grown(self._work, need, self.device, stream, self._kept)
            one = x.shape[0] == 1
            rc = L.lib().bs_lora_add_async(self.ref, batch.dev.data_ptr(), x.shape[0], x.data_ptr(),
                                           self.cols if one else x.stride(0), y.data_ptr(), out.data_ptr(),
                                           self.rows if one else y.stride(0),
                                           L.T_FP32 if y.dtype == torch.float32 else L.T_BF16, self._work.data_ptr(),
                                           self._work.numel(), _stream_of(self.device, stream))
        if rc:
            L.check(rc, "bs_lora_add_async")
        return out


class LoraBatch:
    """Which adapter each token of a step has (bs_lora_batch_async)."""

    def __init__(self, adapter_of: torch.Tensor, adapters: int, stream=None):
        """adapter_of: an int32 device tensor, one index per token, -1 for none;
        adapters: how many the packs hold."""
        if adapter_of.dtype != torch.int32 or adapter_of.dim() != 1 or not adapter_of.is_contiguous():
            raise ValueError("adapter_of must be a contiguous int32 vector")
        self.tokens, self.adapters = int(adapter_of.numel()), int(adapters)
        need = int(L.lib().bs_lora_batch_bytes(self.tokens, self.adapters)) if 1 <= adapters <= 4096 else 0
        with _on(stream):
            self.dev = torch.empty(max(need // 4, 4), dtype=torch.int32, device=adapter_of.device)
        self.update(adapter_of, stream)

    def update(self, adapter_of: torch.Tensor, stream=None) -> None:
        """Another assignment of as many tokens (the buffer stays, as a captured graph needs)."""
        if adapter_of.dtype != torch.int32 or adapter_of.numel() != self.tokens or not adapter_of.is_contiguous():
            raise ValueError(f"adapter_of must be a contiguous int32 vector of {self.tokens}")
        _same_device(self.dev.device, adapter_of=adapter_of)
        rc = L.lib().bs_lora_batch_async(adapter_of.data_ptr(), self.tokens, self.adapters, self.dev.data_ptr(),
                                         4 * self.dev.numel(), _stream_of(adapter_of.device, stream))
        L.check(rc, "bs_lora_batch_async")

    def bad_indices(self) -> int:
        """Indices that named no adapter (they count as none); synchronises."""
        return int(self.dev[2].item())

    def check_for(self, pack: LoraPack, tokens: int) -> None:
        if tokens != self.tokens or pack.adapters != self.adapters:
            raise ValueError(f"a batch of {self.tokens} tokens over {self.adapters} adapters, used for {tokens} tokens "
                             f"over {pack.adapters}")
