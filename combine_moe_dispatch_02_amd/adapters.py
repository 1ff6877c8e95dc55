"""Low-rank adapters of many requests beside one shared projection: their tables, the grouping of a
batch's rows, and the buffers of moe_adapter and moe_adapter_backward (block.py), kept together.

The projection may be any that maps bf16 rows [T, K] to [T, N]; ``StreamMoE`` takes an ``Adapters``
for the layer itself (K = N = H). Several projections of one batch share a grouping.
"""
from __future__ import annotations

from typing import Optional

import torch

from .block import (adapter_backward_workspace_bytes, adapter_tile, adapter_workspace_bytes, moe_adapter,
                    moe_adapter_backward)
from .layer import Plan, Workspace, moe_plan

__all__ = ["AdapterRows", "Adapters"]


class AdapterRows:
    """Which adapter each of a batch's rows has: ``ids`` int32 [T], -1 (or any id outside
    [begin, begin + n)) for none. ``set`` is called once for a batch, before its projections; without
    gradients up to 64 rows need no more than the ids, others are grouped by moe_plan. ``ids`` is read by set() in the second case
    and by every later call in the first: it is left unchanged until the batch is done. One batch at a time, in graphs too."""

    def __init__(self, T: int, n: int, *, begin: int = 0, train: bool = False, device="cuda", tile: Optional[int] = None):
        self.T, self.n, self.begin = T, n, begin
        self.ids: Optional[torch.Tensor] = None
        self.batch = 0                # how often set() has grouped rows
        self.plan: Optional[Plan] = None
        if T > 64 or (train and T > 0):
            tile = adapter_tile(T, n) if tile is None else tile
            self.plan = Plan.allocate(T, 1, begin, n, tile, device)
            self._ws = Workspace(T, 1, n, tile, device=device)

    def set(self, ids: torch.Tensor, stream=None) -> "AdapterRows":
        if ids.shape != (self.T,) or ids.dtype != torch.int32:
            raise ValueError(f"ids must be int32 [{self.T}]")
        if self.plan is not None:
            if ids.device != self.plan.pos.device:
                raise ValueError(f"ids are on device {ids.device}, the rows on {self.plan.pos.device}")
            with torch.cuda.device_of(ids):          # need not be the current one
                moe_plan(ids.view(self.T, 1), self.plan, self._ws, stream)
        self.ids = ids
        self.batch += 1
        return self

    def by(self) -> dict:
        """How moe_adapter is told of the rows."""
        if self.ids is None:
            raise RuntimeError("AdapterRows.set() has not been called")
        return {"plan": self.plan} if self.plan is not None else {"ids": self.ids, "id_begin": self.begin}


class Adapters:
    """a bf16 [n, R, K], b bf16 [n, N, R], scale fp32 [n], ranks int32 [n] (both optional) of one projection,
    for batches of ``rows`` (an AdapterRows). With train=True, ``add`` keeps what ``backward`` takes, and ``da`` and
    ``db`` (fp32) receive the gradients. All calls share the workspaces, v, da and db: one at a time, in graphs too, and of
    several ``add`` calls the last has its gradients; layers that run at once, or whose backward passes come after both forward
    passes, have an Adapters each."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, rows: AdapterRows, *, scale: Optional[torch.Tensor] = None,
                 ranks: Optional[torch.Tensor] = None, train: bool = False):
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("a must be [n, R, K], b [n, N, R]")
        if a.shape[0] != rows.n:
            raise ValueError(f"{a.shape[0]} adapters, the rows are of {rows.n}")
        if train and rows.T > 0 and rows.plan is None:
            raise ValueError("gradients need AdapterRows(train=True)")
        self.a, self.b, self.rows, self.scale, self.ranks, self.train = a, b, rows, scale, ranks, train
        self.added = 0                # calls of add()
        (n, R, K), N = a.shape, b.shape[1]
        u8 = dict(dtype=torch.uint8, device=a.device)
        self._ws = torch.empty(adapter_workspace_bytes(rows.T, K, R), **u8)
        if train:
            self._bws = torch.empty(adapter_backward_workspace_bytes(rows.T, n, K, N, R), **u8)
            self.v = torch.empty(rows.T, R, dtype=torch.float32, device=a.device)
            self.da = torch.empty(n, R, K, dtype=torch.float32, device=a.device)
            self.db = torch.empty(n, N, R, dtype=torch.float32, device=a.device)
            self._x: Optional[torch.Tensor] = None
            self._batch = 0           # that of the rows which v is of

    def add(self, x: torch.Tensor, base: Optional[torch.Tensor], out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """out = base + each row's adapter of x; out None: in place, into base."""
        out = base if out is None else out
        moe_adapter(x, self.a, self.b, out, self._ws, base=base, scale=self.scale, ranks=self.ranks,
                    v=self.v if self.train else None, stream=stream, **self.rows.by())
        self.added += 1
        if self.train:
            self._x, self._batch = x, self.rows.batch
        return out

    def check_backward(self) -> None:
        if not self.train or self._x is None:
            raise RuntimeError("no add() with train=True to take the gradients of")
        if self._batch != self.rows.batch:
            raise RuntimeError("AdapterRows.set() has grouped other rows since the add() whose gradients these would be")

    def backward(self, dout: torch.Tensor, dx_base: Optional[torch.Tensor], dx: Optional[torch.Tensor] = None, stream=None) -> None:
        """da, db and dx = dx_base + the adapters' share (dx None: in place, into dx_base; both None: no dx) for the last
        ``add``, whose x must hold what it held and whose rows must not have been set again since (with graphs:
        both captured, or neither)."""
        self.check_backward()
        dx = dx_base if dx is None else dx
        moe_adapter_backward(dout, self._x, self.v, self.a, self.b, self.rows.plan, self._bws, self.da, self.db, dx,
                             dx_base=dx_base, scale=self.scale, ranks=self.ranks, stream=stream)
